"""Host-side rules and refusals of the operators around the decode step that
need no GPU, beyond those of test_serving_cpu.py."""
import ctypes
import os
import shutil
import subprocess

import pytest

from mlra_latent_kv_b200 import abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_prompt_takes_the_cuda_core_kernel_where_the_other_was_compiled_otherwise(tmp_path):
    src, exe = tmp_path / "path.cc", str(tmp_path / "path")
    src.write_text("""
#include "prompt_path.h"
using namespace mlra;
#define IS(kernel, fits, regs, path) if (prompt_path(kernel, fits, regs, 168) != PromptPath::path) return __LINE__;
int main() {
  IS(MLRA_KERNEL_AUTO, true, 168, kTc)
  IS(MLRA_KERNEL_TC, true, 168, kTc)
  IS(MLRA_KERNEL_AUTO, true, 160, kSimt)
  IS(MLRA_KERNEL_AUTO, true, 255, kSimt)
  IS(MLRA_KERNEL_TC, true, 160, kNoRegisters)
  IS(MLRA_KERNEL_AUTO, false, 0, kSimt)
  IS(MLRA_KERNEL_TC, false, 0, kNoShape)
  IS(MLRA_KERNEL_SIMT, true, 168, kSimt)
  IS(MLRA_KERNEL_SIMT, false, 0, kSimt)
}
""")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", "/usr/local/cuda/include", "-I",
                        os.path.join(ROOT, "mlra_latent_kv_b200", "csrc"), str(src), "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe]).returncode == 0


def _dims(**kw):
    return abi.make_dims(**(dict(B=2, H=8, d_h=128, d_v=128, d_c=512, d_r=64, max_pages_per_seq=8, num_pages=32) | kw))


def test_binding_refuses_numbers_that_do_not_fit(L):
    """2^32 + 5 would be 5 in the library's 32 bits."""
    d = _dims()
    need = abi.prompt_workspace_bytes(d, 100, 100, 8)
    for sizes in ((2 ** 32 + 100, 100, 8), (100, 2 ** 32 + 100, 8), (100, 100, 2 ** 32 + 8), (-2 ** 32 + 100, 100, 8)):
        with pytest.raises(abi.MlraError, match="out of range"):
            abi.prompt_workspace_bytes(d, *sizes)
    assert abi.prompt_workspace_bytes(d, 100, 100, 8) == need
    for recent in (2 ** 32 + 5, 2 ** 31, -2 ** 32):
        with pytest.raises(abi.MlraError, match="recent"):
            abi.latent_evict(d, recent, *[None] * 10)
    with pytest.raises(TypeError):  # not a whole number
        abi.latent_evict(d, 16.5, *[None] * 10)


FAR = 1 << 34  # fake buffers this far apart do not overlap


def _status(fn, head, names, at, ws):
    """fn with fake buffers far from one another, but for `at` = (one of them, another, bytes behind its start)."""
    p = {n: FAR * (i + 1) for i, n in enumerate(names)}
    p[at[0]] = p[at[1]] + at[2]
    return fn(*head, *p.values(), ws, None)


PROMPT = ("q_nope", "q_rope", "cu_q", "k_nope", "v", "cu_k", "rope_cache", "page_table", "out", "lse", "workspace")


@pytest.mark.parametrize("out", ["out", "lse", "workspace"])
def test_prompt_refuses_outputs_over_inputs(L, out):
    d = _dims(kernel="simt")  # which asks no device before it looks
    s = abi.PromptShape(8, 100, 100, (8 * 200, 200), (8 * 64, 64), (8 * 128, 128), (8 * 128, 128))
    for name in PROMPT:
        if name != out:
            at = (out, name, 0)
            assert _status(L.mla_prompt, (ctypes.byref(d), ctypes.byref(s)), PROMPT, at, 1 << 20) == 1
            assert "overlap" in abi.last_error()
    # the last byte of a strided input: 99 tokens and 7 heads of 200, then 128 columns of two bytes
    end = ((99 * 8 + 7) * 200 + 128) * 2
    assert end % 16 == 0
    assert _status(L.mla_prompt, (ctypes.byref(d), ctypes.byref(s)), PROMPT, ("out", "q_nope", end - 16),
                   1 << 20) == 1 and "overlap" in abi.last_error()


def test_absorb_and_weights_refuse_outputs_over_inputs(L):
    d = _dims()
    names = ("q_nope", "q_rope", "q_pos", "W_UK", "q_abs", "workspace")
    for out in ("q_abs", "workspace"):
        for name in names:
            if name != out:
                assert _status(L.mlra_absorb, (ctypes.byref(d),), names, (out, name, 0), 256) == 1
                assert "overlap" in abi.last_error()
    names = ("q_abs", "lse", "latent_cache", "rope_cache", "page_table", "seq_lens", "weights_in", "weights", "workspace")
    for out in ("weights", "workspace"):
        for name in names:
            if name != out and (out, name) != ("weights", "weights_in"):
                assert _status(L.mlra_attention_weights, (ctypes.byref(d),), names, (out, name, 0), 256) == 1
                assert "overlap" in abi.last_error()


def test_evict_refuses_a_workspace_over_its_buffers(L):
    d = _dims()
    names = ("evict_pages", "weights", "page_table", "seq_lens", "latent_cache", "rope_cache", "weights_out",
             "page_table_out", "seq_lens_out", "workspace")
    for name in names[:-1]:
        assert _status(L.latent_evict, (ctypes.byref(d), 0), names, ("workspace", name, 0), 1 << 20) == 1
        assert "overlap" in abi.last_error()
