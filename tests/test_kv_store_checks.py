"""The bounds-checked build covers the paged-cache kernels: every store of theirs to an output,
a page or a partial sum goes through the checked store (CPU: read from the sources), and each
form gives oracle parity with no bounds status on that build (GPU)."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_layer_residual_b200", "csrc")
RAW = [r"__stcg\(", r"\*\s*reinterpret_cast<[^>;]*>\([^;]*\)\s*=(?!=)", r"\bdst\[[^\];]*\]\s*=(?!=)",
       r"\bp\.(?!counters)\w+\[[^;]*\]\s*=(?!=)", r"\(is_v \?[^;]*\)\[[^;]*\]\s*=(?!=)"]


@pytest.mark.parametrize("name", ["k7_kv.cuh", "k8_attend.cuh", "k9_prompt.cuh"])
def test_every_store_is_a_checked_one(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    raw = [m.group(0) for pattern in RAW for m in re.finditer(pattern, text)]
    assert not raw, raw
    assert "kv_store" in text


def _child():
    """Runs in the child process: FNL_LIBRARY=debug is already set."""
    sys.path.insert(0, ROOT)
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    import test_gpu_kv as t
    from kv_cases import Cache
    from transformer_layer_residual_b200 import fnl

    assert fnl.lib_path().endswith("libfnl_debug.so"), fnl.lib_path()
    h = fnl.Handle(0)
    with open("/proc/self/maps") as f:
        assert "libfnl_debug.so" in f.read(), "the debug build is not the loaded library"
    for fmt in ("bf16", "int4"):
        for D, page, Hq, Hkv in ((64, 16, 4, 2), (128, 64, 14, 2)):
            for rot, interleaved in ((0, False), (64, False), (48, True)):
                t.test_append(h, fmt, rot, interleaved, D, page, Hq, Hkv)
            for heads in (4, 8):      # 8 and 16 rows a key head; whole heads and parts, empty sequences, rows behind
                c = Cache(fmt, [1, 33, 0, 129, 3000], 2, D, page, seed=D)
                assert "split" in t._check_attention(h, c, [1, 2, 0, 1, 2], 2 * heads)
            c = Cache(fmt, [1, 65, 40, 255, 3000, 300], 2, D, page, seed=D + 1)
            for window, sinks in ((0, 0), (200, 33)):
                assert "tensor" in t._check_attention(h, c, [1, 65, 0, 127, 20, 300], 6, window, sinks)
            print(fmt, D, "ok", flush=True)
        t.test_strided_pages(h)
    h.check()
    h.close()


@pytest.mark.gpu
def test_debug_build_parity_no_bounds_status(cuda_device):
    lib = os.path.join(ROOT, "transformer_layer_residual_b200", "libfnl_debug.so")
    if not os.path.exists(lib):
        pytest.fail(f"{lib} is missing: build it with python -m transformer_layer_residual_b200.build --debug")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=dict(os.environ, FNL_LIBRARY="debug"), cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    print(r.stdout[-4000:])
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


if __name__ == "__main__":
    _child()
