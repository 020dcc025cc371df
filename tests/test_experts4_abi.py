"""include/moe_experts4.h: every declared entry point is exported, bound and refuses a null handle before any device
work; the binding's shapes follow the header's layout (no GPU needed)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared():
    text = open(os.path.join(ROOT, "include", "moe_experts4.h")).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*int\s+(moex4_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_entry_point_is_exported_and_bound():
    import load_balance_planning_amd as m
    lib = m.lib()
    out = subprocess.run(["nm", "-D", "--defined-only", m.lib_path()], capture_output=True, text=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert len(declared()) == 7
    assert set(declared()) <= exported
    assert set(m.EXPERT4_EXPORTS) == set(declared())
    for name in declared():
        assert callable(getattr(m, name)) and getattr(lib, name).argtypes is not None, name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "moe_experts4.h"\nint main(void) { return moex4_quantize == 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-Wno-address", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def test_a_null_handle_is_refused():
    import load_balance_planning_amd as m
    lib = m.lib()
    calls = {
        "moex4_quantize": (None, None, 1, 1, None, None, None),
        "moex4_quantize_weights": (None, None, 1, 1, 1, None, None, None, None, None),
        "moex4_values": (None, None, None, 1, 1, 1, None, None),
        "moex4_swiglu": (None, None, 1, 1, None, None, None),
        "moex4_matmul": (None, None, None, 4, None, None, None, None, 1, 1, None, None),
        "moex4_experts_work": (None, 1, None),
        "moex4_experts": (None, None, None, None, 4, 1) + (None,) * 7,
    }
    assert set(calls) == set(declared())
    for name, args in calls.items():
        assert getattr(lib, name)(*args) == m.MOE_ERR_INVALID_ARG, name


@pytest.mark.parametrize("cols,padded", [(1, 256), (256, 256), (257, 512), (2048, 2048), (2688, 2816), (7168, 7168)])
def test_shapes(cols, padded):
    import load_balance_planning_amd as m
    assert m.Blocks4.padded(cols) == padded
    assert m.Blocks4.shapes((5,), cols) == ((5, padded // 2), (padded // 256, 5, 8))
    assert m.Blocks4.shapes((3, 5), cols) == ((3, 5, padded // 2), (3, padded // 256, 5, 8))


def test_the_binding_names_the_scales_types():
    import load_balance_planning_amd as m
    assert (m.BLOCK4, m.LINE4, m.FEW_TOKENS) == (32, 256, 64)
