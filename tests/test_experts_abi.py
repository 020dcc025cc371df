"""include/moe_experts.h: every declared entry point is exported, bound and refuses a null handle
before any device work, and the binding's sizes follow the header's layout (no GPU needed)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared():
    text = open(os.path.join(ROOT, "include", "moe_experts.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*int\s+(moex_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_entry_point_is_exported_and_bound():
    import load_balance_planning_amd as m
    lib = m.lib()
    out = subprocess.run(["nm", "-D", "--defined-only", m.lib_path()], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert len(declared()) == 10
    assert set(declared()) <= exported
    assert set(m.EXPERT_EXPORTS) == set(declared())
    for name in declared():
        assert callable(getattr(m, name)) and getattr(lib, name).argtypes is not None, name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { moex_gate_config g = {MOEX_SIGMOID, 8, 4, 2, 1, 2.5f};'
                   ' return g.n_group == 8 ? 0 : 1; }\n')
    exe = tmp_path / "use"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_a_null_handle_is_refused():
    import load_balance_planning_amd as m
    lib = m.lib()
    calls = {
        "moex_gate": (None,) * 8,
        "moex_gate_grad": (None,) * 7,
        "moex_quantize": (None, None, 1, 1, None, None, None),
        "moex_quantize_weights": (None, None, 1, 1, 1, None, None, None, None, None),
        "moex_swiglu": (None, None, 1, 1, None, None, None),
        "moex_swiglu_grad": (None, None, None, 1, 1, None, None, None),
        "moex_matmul": (None,) * 7 + (1, 1, None, None),
        "moex_wgrad": (None,) * 7 + (1, 1, None, None),
        "moex_combine": (None,) * 6,
        "moex_combine_grad": (None,) * 8,
    }
    assert set(calls) == set(declared())
    for name, args in calls.items():
        assert getattr(lib, name)(*args) == m.MOE_ERR_INVALID_ARG, name


@pytest.mark.parametrize("cols,padded,scales", [(1, 128, 4), (128, 128, 4), (129, 256, 4), (512, 512, 4),
                                                (513, 640, 8), (2688, 2688, 24), (7168, 7168, 56)])
def test_block_sizes(cols, padded, scales):
    import load_balance_planning_amd as m
    assert (m.Blocks.padded(cols), m.Blocks.scales(cols)) == (padded, scales)


def test_make_gate():
    import load_balance_planning_amd as m
    g = m.make_gate("sigmoid", 8, 4, 2, True, 2.5)
    assert (g.score, g.n_group, g.topk_group, g.group_top, g.renorm, g.scale) == (1, 8, 4, 2, 1, 2.5)
    with pytest.raises(ValueError):
        m.make_gate("relu")
