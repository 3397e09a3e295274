"""Host-side checks of the prompt and eviction operators (include/mlra_serving.h)
that need no GPU: the header from C, the refusals of bad arguments before
anything is enqueued (fake device pointers are never dereferenced on these
paths), and the 64-bit forms against brute force."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from mlra_latent_kv_b200 import abi, build
from oracle import serving as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
FAR = 1 << 34  # fake buffers that do not overlap


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def _dims(**kw):
    base = dict(B=2, H=8, d_h=128, d_v=128, d_c=512, d_r=64, max_pages_per_seq=8, num_pages=32)
    base.update(kw)
    return abi.make_dims(**base)


def _shape(d, kv=8, tq=100, tk=100, **over):
    s = abi.PromptShape(kv, tq, tk, (d.H * d.d_h, d.d_h), (d.H * d.d_r, d.d_r), (kv * d.d_h, d.d_h),
                        (kv * d.d_v, d.d_v))
    for k, v in over.items():
        getattr(s, k)[:] = v
    return s


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c_consumer_compiles_links_and_validates(tmp_path, L):
    libdir, exe = os.path.dirname(build.LIB), str(tmp_path / "serving_consumer")
    src = os.path.join(ROOT, "tests", "serving_consumer.c")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                        "/usr/local/cuda/include", src, "-L", libdir, "-lmlra", f"-Wl,-rpath,{libdir}", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout + run.stderr
    header = open(os.path.join(ROOT, "include", "mlra_serving.h")).read()
    names = re.findall(r"MLRA_SERVING_API\s+[\w\s\*]+?\b(\w+)\s*\(", header)
    assert run.stdout.startswith(f"ok {len(names)} entry points")
    for n in names:
        assert f"(void*){n}" in open(src).read() and n in abi.SIGNATURES


def _prompt(L, d, s, ws=1 << 40, **over):
    args = dict(q_nope=FAKE, q_rope=FAKE, cu_q=FAKE, k_nope=FAKE, v=FAKE, cu_k=FAKE, rope_cache=FAKE,
                page_table=FAKE, out=FAKE, lse=None, workspace=FAKE) | over
    return L.mla_prompt(ctypes.byref(d), ctypes.byref(s) if s else None, *args.values(), ws, None)


@pytest.mark.parametrize("over,status", [
    (dict(kv=3), 1), (dict(kv=0), 1), (dict(tq=-1), 1), (dict(tk=-1), 1), (dict(q_nope_stride=(-8, 128)), 1),
    (dict(v_stride=(1024, 64)), 1), (dict(k_nope_stride=(0, 128)), 1), (dict(q_rope_stride=(1 << 40, 64)), 1),
])
def test_prompt_shape_refusals(L, over, status):
    d = _dims()
    s = _shape(d, **over)
    assert L.mla_prompt_workspace_bytes(ctypes.byref(d), ctypes.byref(s)) == 0
    assert _prompt(L, d, s) == status and abi.last_error()


@pytest.mark.parametrize("dims,status", [(dict(n_branch=4), 1), (dict(d_v=516), 2), (dict(d_r=3), 1),
                                         (dict(dtype="f32", kernel="tc"), 2), (dict(d_h=64, kernel="tc"), 2)])
def test_prompt_dims_refusals(L, dims, status):
    d = _dims(**dims)
    assert _prompt(L, d, _shape(d)) == status


def test_prompt_pointer_refusals(L):
    d = _dims()
    s = _shape(d)
    assert _prompt(L, d, None) == 1
    for name in ("q_nope", "q_rope", "cu_q", "k_nope", "v", "cu_k", "rope_cache", "page_table", "out", "workspace"):
        assert _prompt(L, d, s, **{name: None}) == 1 and name in abi.last_error()
    assert _prompt(L, d, s, out=FAKE + 8) == 1
    assert _prompt(L, d, s, cu_q=FAKE + 2) == 1
    assert _prompt(L, d, s, lse=FAKE + 2) == 1
    assert _prompt(L, d, s, workspace=FAKE + 16) == 1
    need = L.mla_prompt_workspace_bytes(ctypes.byref(d), ctypes.byref(s))
    assert _prompt(L, d, s, ws=need - 1) == 3
    assert _prompt(L, d, _shape(d, tq=0), q_nope=None) == 0  # no rows: nothing to do


def test_absorb_refusals(L):
    d = _dims()
    ok = dict(q_nope=FAKE, q_rope=FAKE, q_pos=FAKE, W_UK=FAKE, q_abs=FAKE, workspace=FAKE)
    call = lambda ws=256, **o: L.mlra_absorb(ctypes.byref(d), *(ok | o).values(), ws, None)  # noqa: E731
    for name in ok:
        assert call(**{name: None}) == 1 and name in abi.last_error()
    assert call(W_UK=FAKE + 8) == 1
    assert call(ws=255) == 3
    d = _dims(kernel="tc", d_h=96)
    assert call() == 2


def test_weights_refusals(L):
    d = _dims(kernel="tc", dtype="f32")
    ok = dict(q_abs=FAKE, lse=FAKE, latent=FAKE, rope=FAKE, table=FAKE, lens=FAKE, weights_in=FAKE, weights=FAKE,
              workspace=FAKE)
    call = lambda ws=256, **o: L.mlra_attention_weights(ctypes.byref(d), *(ok | o).values(), ws, None)  # noqa: E731
    assert call() == 2
    d = _dims()
    for name in ok:
        if name != "weights_in":
            assert call(**{name: None}) == 1
    assert call(weights_in=FAKE + 2) == 1
    assert call(weights_in=FAKE + 4) == 1 and "overlap" in abi.last_error()
    assert call(ws=255) == 3


def test_evict_refusals(L):
    d = _dims()
    names = ("evict_pages", "weights", "page_table", "seq_lens", "latent_cache", "rope_cache", "weights_out",
             "page_table_out", "seq_lens_out")
    ok = {n: FAR * (i + 1) for i, n in enumerate(names)} | {"workspace": FAKE}
    need = abi.evict_workspace_bytes(d)
    call = lambda recent=0, ws=need, **o: L.latent_evict(  # noqa: E731
        ctypes.byref(d), recent, *(ok | o).values(), ws, None)
    for name in ok:
        assert call(**{name: None}) == 1 and name in abi.last_error()
    assert call(recent=-1) == 1
    assert call(ws=need - 1) == 3
    assert call(weights_out=ok["weights"]) == 1 and "overlaps an input" in abi.last_error()
    assert call(page_table_out=ok["page_table"] + 4) == 1
    assert call(seq_lens_out=ok["weights_out"] + 4) == 1 and "two outputs" in abi.last_error()
    # error record | owners | counts | two lists of 32 slots per table entry
    r = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert need == r(256 + 32 * 4) + r(2 * 4) + 2 * r(2 * 8 * 32 * 4)
    assert L.latent_evict_workspace_bytes(ctypes.byref(_dims(page_size=32))) == 0


def test_binding_refuses_host_tensors():
    d = _dims()
    with pytest.raises(abi.MlraError, match="CUDA tensor"):
        abi.absorb_query(d, *[torch.zeros(1)] * 6)
    with pytest.raises(abi.MlraError, match=r"\[tokens, heads, width\]"):
        abi.mla_prompt(d, torch.zeros(4, 8), *[torch.zeros(1)] * 9)


# ---------------------------------------------------------------------------
# the 64-bit forms themselves
# ---------------------------------------------------------------------------
def test_prompt_form_matches_the_unabsorbed_decode_row_by_row():
    """Its last row is the decode of that token, and it is causal: a longer prompt repeats a shorter one's rows."""
    rng = np.random.default_rng(0)
    n, H, d_h, d_r, d_v = 70, 2, 8, 4, 6
    q, qr = rng.standard_normal((n, H, d_h)), rng.standard_normal((n, H, d_r))
    k, v = rng.standard_normal((n, 1, d_h)), rng.standard_normal((n, 1, d_v))
    raw = rng.standard_normal((n, d_r))
    pool = np.zeros((3, 64, d_r))
    row = np.array([[2, 0]])
    rot = ref.rope(raw, np.arange(n))
    pool[2], pool[0, :6] = rot[:64], rot[64:]
    out, lse, *_ = ref.prompt(q, qr, [0, n], k, v, [0, n], pool, row, 0.3)
    for h in range(H):
        x = 0.3 * (k[:, 0] @ q[-1, h] + ref.rope(raw, np.arange(n)) @ ref.rope(qr[-1, h], n - 1))
        p = np.exp(x) / np.exp(x).sum()
        np.testing.assert_allclose(out[-1, h], p @ v[:, 0], rtol=1e-12)
        np.testing.assert_allclose(lse[-1, h], np.log2(np.exp(x).sum()), rtol=1e-12)
    short, *_ = ref.prompt(q[:20], qr[:20], [0, 20], k[:20], v[:20], [0, 20], pool, row, 0.3)
    np.testing.assert_allclose(short, out[:20], rtol=1e-12)
    # more queries than keys: the first have none
    few, none, *_ = ref.prompt(q[:5], qr[:5], [0, 5], k[:2], v[:2], [0, 2], pool, row, 0.3)
    assert (few[:3] == 0).all() and np.isneginf(none[:3]).all() and np.isfinite(none[3:]).all()


def test_weights_form_sums_to_one_per_head_and_branch():
    rng = np.random.default_rng(1)
    n, H, d_c, d_r, nb = 100, 3, 8, 4, 2
    pool, rope = rng.standard_normal((2, 64, d_c)), rng.standard_normal((2, 64, d_r))
    q = rng.standard_normal((1, H, d_c + d_r))
    lse = np.zeros((1, nb, H))
    c, k = ref.cached(pool, [1, 0], n), ref.cached(rope, [1, 0], n)
    for r in range(nb):
        s = np.concatenate((c[:, 4 * r:4 * r + 4], k), 1) @ \
            np.concatenate((q[0][:, 4 * r:4 * r + 4], q[0][:, d_c:]), 1).T
        lse[0, r] = np.log2(np.exp2(s).sum(0))
    (p, _), = ref.weights(q, lse, pool, rope, np.array([[1, 0]]), [n], nb)
    assert p.shape == (n,) and abs(p.sum() - nb * H) < 1e-9
    lse[0, 0, 1] = -np.inf  # a head that attended nothing
    (p, _), = ref.weights(q, lse, pool, rope, np.array([[1, 0]]), [n], nb)
    assert abs(p.sum() - (nb * H - 1)) < 1e-9


def test_evict_form_keeps_the_heaviest_and_the_recent():
    rng = np.random.default_rng(2)
    n, maxp, recent = 300, 6, 50
    w = np.zeros((1, maxp * 64), np.float32)
    w[0, :n] = rng.random(n).round(1)  # many ties
    w[0, 7] = np.nan
    table = np.array([[3, 1, 4, 0, 5, -1]], np.int32)
    (moves, new, row, m), = ref.evict(w, table, [n], [2], recent)
    assert m == n - 128 and list(row) == [4, 0, 5, -1, -1, -1]
    src, dst = [s for s, _ in moves], [t for _, t in moves]
    assert all(s < 128 for s in src) and all(128 <= t < n - recent for t in dst) and len(set(dst)) == len(dst)
    assert 7 not in src
    kept = sorted(set(src) | (set(range(128, n)) - set(dst)))
    gone = sorted(set(range(n)) - set(kept))
    assert len(gone) == 128 and max(gone) < n - recent
    key = lambda t: (-np.inf if np.isnan(w[0, t]) else w[0, t], -t)  # noqa: E731
    assert max(key(t) for t in gone) < min(key(t) for t in kept if t < n - recent)
    np.testing.assert_array_equal(np.sort(new[:m]), np.sort(w[0, kept]))
    assert (new[m:] == 0).all()
