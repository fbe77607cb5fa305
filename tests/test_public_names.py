"""The package's public names: all of them listed, all of them there, and torch imported only once a call needs it."""
import os
import subprocess
import sys

import gemv_tile_pipelined_amd as gt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = [f"{name}_{fmt}" for name in ("quantize_fp8_rows", "quantize_fp8_tiles", "gemm_fp8", "gemm_grouped", "gemm_grouped_dgrad",
                                      "gemm_grouped_wgrad", "gemm_grouped_fp8") for fmt in ("f16", "bf16")]


def test_listed_names_exist():
    assert len(set(gt.__all__)) == len(gt.__all__)
    for name in gt.__all__:
        assert getattr(gt, name) is not None, name


def test_tensor_calls_are_listed():
    assert set(CALLS) <= set(gt.__all__) and set(CALLS) <= set(dir(gt)) and "blocks" in dir(gt)
    names = {}
    exec("from gemv_tile_pipelined_amd import *", names)
    assert set(CALLS) <= set(names)
    assert sorted(gt.blocks.__all__) == sorted(CALLS)


def test_every_tensor_call_is_in_the_library():
    assert set(CALLS) <= set(gt.EXPORTED_SYMBOLS)


def test_package_alone_does_not_import_torch():
    code = "import sys, gemv_tile_pipelined_amd as gt; dir(gt); sys.exit('torch' in sys.modules)"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
