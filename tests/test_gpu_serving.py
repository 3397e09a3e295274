"""Prompt attention, absorbed queries, attention weights and eviction on the
GPU against their plain 64-bit forms (oracle/serving.py), at the lengths and
masks where they can go wrong.

Tolerances are bounds computed per output from the inputs (u = half a step of
the type, 2^-24 for fp32, 2^-8 for bf16):
  - a logit that is a sum of products of exact inputs, added up in fp32 over K
    terms, is off by at most K * 2u32 * sum |q||k| (twice u: a tensor core may
    truncate);
  - bf16 adds its rounding of the rotated query, u16 * sum |q_rot||k| of the
    rotary dims, in mla_prompt (mlra_absorb's output is an input of
    mlra_attention_weights, so nothing is rounded there);
  - a weight e^x / sum e^x whose exponents are off by d changes by a factor
    within e^(2d), and the hardware's exponential adds a few u32;
  - bf16 rounds each weight and the output: u16 * sum p|v| and u16 * |out|.
"""
import numpy as np
import pytest
import torch

from mlra_latent_kv_b200 import abi
from oracle import serving as ref

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
FULL = dict(d_h=128, d_r=64, d_v=128, d_c=512)
TINY = dict(d_h=32, d_r=16, d_v=32, d_c=64)
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(x):
    return x.double().cpu().numpy()


def _rand(g, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype]).cuda()


def _pages(g, lens, maxp, spare=2):
    counts = [-(-n // 64) for n in lens]
    order = torch.randperm(sum(counts) + spare, generator=g).to(torch.int32)
    table, at = torch.full((len(lens), maxp), -1, dtype=torch.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), sum(counts) + spare


def _pool(g, lens, table, total, width, dtype):
    """Random tokens; NaN in every slot that no token uses."""
    pool = torch.randn(total, 64, width, generator=g).to(TORCH[dtype])
    used = torch.zeros(total, 64, dtype=torch.bool)
    for row, n in zip(table.cpu(), lens):
        for p in range(-(-n // 64)):
            used[row[p], :min(64, n - 64 * p)] = True
    pool[~used] = float("nan")
    return pool.cuda()


# ---------------------------------------------------------------------------
# prompt
# ---------------------------------------------------------------------------
class Prompt:
    """One mla_prompt call: packed inputs, a NaN-filled out with rows behind the last sequence."""

    def __init__(self, dtype, q_lens, k_lens, H, kv, seed=0, dims=None, kernel="auto", scale=1.0, pad=3,
                 interleaved=True, offset=0):
        g = torch.Generator().manual_seed(seed)
        w = dims or FULL
        self.dtype, self.H, self.kv, self.w = dtype, H, kv, w
        B, tq, tk = len(q_lens), sum(q_lens) + pad, sum(k_lens) + pad
        if interleaved:  # as the projections leave them
            q = _rand(g, tq, H, w["d_h"] + w["d_r"] + offset, dtype=dtype, scale=scale)
            kvp = _rand(g, tk, kv, w["d_h"] + w["d_v"] + offset, dtype=dtype)
            self.q_nope, self.q_rope = q[..., :w["d_h"]], q[..., w["d_h"]:w["d_h"] + w["d_r"]]
            self.k_nope, self.v = kvp[..., :w["d_h"]], kvp[..., w["d_h"]:w["d_h"] + w["d_v"]]
        else:
            self.q_nope = _rand(g, tq, H, w["d_h"], dtype=dtype, scale=scale)
            self.q_rope = _rand(g, tq, H, w["d_r"], dtype=dtype, scale=scale)
            self.k_nope = _rand(g, tk, kv, w["d_h"], dtype=dtype)
            self.v = _rand(g, tk, kv, w["d_v"], dtype=dtype)
        self.k_nope[sum(k_lens):], self.v[sum(k_lens):] = float("nan"), float("nan")
        cu = lambda n: torch.tensor([sum(n[:i]) for i in range(B + 1)], dtype=torch.int32).cuda()  # noqa: E731
        self.cu_q, self.cu_k = cu(q_lens), cu(k_lens)
        self.maxp = max(1, -(-max(k_lens) // 64)) + 1
        self.table, total = _pages(g, k_lens, self.maxp)
        self.rope_cache = _pool(g, k_lens, self.table, total, w["d_r"], dtype)
        self.dims = abi.make_dims(B=B, H=H, max_pages_per_seq=self.maxp, num_pages=total, dtype=dtype, kernel=kernel,
                                  **w)
        self.scale = (w["d_h"] + w["d_r"]) ** -0.5
        self.ws = torch.zeros(abi.prompt_workspace_bytes(self.dims, tq, tk, kv), dtype=torch.uint8, device="cuda")
        self.out = torch.full((tq, H, w["d_v"]), float("nan"), dtype=TORCH[dtype], device="cuda")
        self.lse = torch.full((tq, H), float("nan"), device="cuda")

    def call(self, lse=True, stream=None, out=None):
        abi.mla_prompt(self.dims, self.q_nope, self.q_rope, self.cu_q, self.k_nope, self.v, self.cu_k,
                       self.rope_cache, self.table, self.out if out is None else out, self.ws,
                       lse=self.lse if lse else None, stream=stream)

    def check(self):
        abi.check_status(self.ws)
        n = int(self.cu_q[-1])
        out, lse, spread, rot, dot = ref.prompt(_np(self.q_nope), _np(self.q_rope), self.cu_q.tolist(),
                                                _np(self.k_nope), _np(self.v), self.cu_k.tolist(),
                                                _np(self.rope_cache), self.table.cpu().numpy(), self.scale)
        got, got_lse = _np(self.out), _np(self.lse)
        K = self.w["d_h"] + self.w["d_r"] + 4           # + 4: the rotation's own roundings
        off = 2 * K * U32 * dot
        if self.dtype == "bf16":
            off = off + U16 * rot
        keys = float((self.cu_k[1:] - self.cu_k[:-1]).max())
        tol = (np.expm1(2 * off)[..., None] + (2 * keys + 16) * U32) * spread + 1e-30
        if self.dtype == "bf16":
            tol = tol * (1 + U16) + U16 * spread * (1 + U16) + U16 * np.abs(out)
        assert np.isfinite(got[:n]).all()
        worst = (np.abs(got[:n] - out[:n]) / tol[:n]).max()
        assert worst <= 1, f"{worst:.2f} of the bound"
        assert np.isnan(got[n:]).all(), "rows behind the last sequence were written"
        some = np.isfinite(lse[:n])
        assert np.isneginf(got_lse[:n][~some]).all()
        # log2 of a sum of `keys` terms, each within e^off
        tol = off[:n] * ref.LOG2E + (keys + 16) * U32 * ref.LOG2E + 4 * U32 * np.abs(np.where(some, lse[:n], 0))
        assert (np.abs(got_lse[:n] - lse[:n])[some] <= tol[some]).all()
        assert np.isnan(got_lse[n:]).all()


RAGGED = [(0, 1, 2, 63, 64, 65), (127, 128, 129, 1), (255, 256, 257), (300,)]


@pytest.mark.parametrize("lens", RAGGED)
@pytest.mark.parametrize("dtype,dims,H,kv", [("f32", TINY, 8, 8), ("f32", TINY, 6, 2), ("bf16", TINY, 3, 1),
                                             ("bf16", FULL, 4, 4), ("bf16", FULL, 8, 2), ("bf16", FULL, 6, 2),
                                             ("f32", FULL, 2, 1)])
def test_prompt_ragged(dtype, dims, H, kv, lens):
    p = Prompt(dtype, lens, lens, H, kv, dims=dims)
    p.call()
    p.check()


@pytest.mark.parametrize("q_lens,k_lens", [((1, 1, 1), (1, 200, 64)), ((5, 130, 64), (517, 131, 64)),
                                           ((1, 257), (1000, 700)), ((3, 0, 200), (3, 40, 0)), ((70, 9), (20, 8))])
@pytest.mark.parametrize("dtype,H,kv", [("f32", 3, 3), ("bf16", 3, 3), ("bf16", 16, 2), ("bf16", 128, 1)])
def test_prompt_behind_a_context_and_rows_without_keys(dtype, H, kv, q_lens, k_lens):
    p = Prompt(dtype, q_lens, k_lens, H, kv, dims=FULL if dtype == "bf16" else TINY, seed=1)
    p.call()
    p.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d_h,d_r,d_v", [(512, 64, 32), (512, 64, 100), (40, 6, 300), (512, 64, 512), (5, 2, 3)])
def test_prompt_other_widths(dtype, d_h, d_r, d_v):
    p = Prompt(dtype, (70, 1, 150), (170, 90, 150), 2, 1, dims=dict(d_h=d_h, d_r=d_r, d_v=d_v, d_c=64), seed=10)
    p.call()
    p.check()


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_prompt_flat_and_peaked(scale):
    p = Prompt("bf16", (150, 300), (150, 400), 4, 4, scale=scale, seed=2)
    p.call()
    p.check()


@pytest.mark.parametrize("interleaved,offset", [(False, 0), (True, 8), (True, 1)])
def test_prompt_strides(interleaved, offset):
    """Dense inputs, views with a gap, views whose rows are not 16-byte aligned."""
    p = Prompt("bf16", (40, 200), (140, 200), 4, 2, interleaved=interleaved, offset=offset, seed=3)
    p.call()
    p.check()


def test_prompt_heads_first_layout():
    """Tokens inside heads: a head's stride is larger than a token's."""
    p = Prompt("bf16", (40, 200), (140, 200), 4, 2, interleaved=False, seed=3)
    for name in ("q_nope", "q_rope", "k_nope", "v"):
        x = getattr(p, name)
        setattr(p, name, x.transpose(0, 1).contiguous().transpose(0, 1))
    assert p.k_nope.stride(1) > p.k_nope.stride(0)
    p.call()
    p.check()


def test_prompt_rising_scores():
    """Each key's score far above all before it: the running maximum moves in every step."""
    p = Prompt("bf16", (600,), (600,), 2, 2, seed=4)
    p.q_nope[:] = 1.0
    p.k_nope[:600] = (torch.arange(600, device="cuda") // 4 / 8.0)[:, None, None]
    p.call()
    p.check()


def test_prompt_without_lse_and_twice_gives_the_same_bits():
    p = Prompt("bf16", (130, 7, 300), (130, 70, 300), 8, 8, seed=5)
    p.call(lse=False)
    assert torch.isnan(p.lse).all()
    first = p.out.clone()
    p.call()
    assert torch.equal(first.view(torch.int16), p.out.view(torch.int16))
    p.check()


def test_prompt_captured_and_on_another_stream():
    p = Prompt("bf16", (130, 7, 300), (130, 70, 300), 8, 8, seed=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.call(stream=s)
    torch.cuda.synchronize()
    want = p.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call()
    p.out.fill_(float("nan"))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), p.out.view(torch.int16))
    p.cu_q.copy_(torch.tensor([0, 1, 1, 200], dtype=torch.int32))  # other lengths, the same graph
    p.cu_k.copy_(torch.tensor([0, 130, 200, 500], dtype=torch.int32))
    p.out.fill_(float("nan"))
    p.lse.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_offsets_out_of_range_are_reported(dtype):
    p = Prompt(dtype, (50, 60, 70), (50, 60, 70), 2, 2, dims=FULL if dtype == "bf16" else TINY, seed=7)
    p.call()
    want = p.out.clone()
    p.out.fill_(float("nan"))
    p.cu_q[3] = 10000  # the last sequence's queries end outside the array
    p.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(p.ws)
    assert torch.equal(p.out[:110], want[:110]) and torch.isnan(p.out[110:].float()).all()
    abi.check_status(p.ws)  # and cleared


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_bad_offset_between_good_ones(dtype):
    p = Prompt(dtype, (50, 60, 70, 40), (50, 60, 70, 40), 2, 2, dims=FULL if dtype == "bf16" else TINY, seed=7)
    p.call()
    want = p.out.clone()
    p.out.fill_(float("nan"))
    p.ws.zero_()
    p.cu_q[2] = 10000  # the second and the third sequence have no rows
    p.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(p.ws)
    for rows in (slice(0, 50), slice(180, 220)):
        assert torch.equal(p.out[rows], want[rows])
    assert torch.isnan(p.out[50:180].float()).all() and torch.isnan(p.out[220:].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_overlapping_sequences_are_reported(dtype):
    p = Prompt(dtype, (50, 60, 70), (50, 60, 70), 2, 2, dims=FULL if dtype == "bf16" else TINY, seed=7)
    p.cu_q[:] = torch.tensor([0, 180, 0, 180], dtype=torch.int32)  # the third goes over the first one's rows again
    p.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(p.ws)


def test_prompt_bad_page_is_reported():
    for dtype, dims in (("f32", TINY), ("bf16", FULL)):
        p = Prompt(dtype, (50, 100), (50, 100), 2, 2, dims=dims, seed=8)
        p.table[1, 1] = 10 ** 6
        p.call()
        with pytest.raises(abi.MlraError):
            abi.check_status(p.ws)


# ---------------------------------------------------------------------------
# absorbed queries
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,dims,B,H", [("f32", TINY, 3, 8), ("bf16", FULL, 1, 5), ("bf16", FULL, 17, 128),
                                            ("bf16", TINY, 5, 3), ("bf16", FULL, 300, 2),
                                            ("bf16", dict(FULL, d_h=64), 100, 2), ("bf16", dict(FULL, d_r=62), 9, 2)])
def test_absorb(dtype, dims, B, H):
    g = torch.Generator().manual_seed(B)
    q, r = _rand(g, B, H, dims["d_h"], dtype=dtype), _rand(g, B, H, dims["d_r"], dtype=dtype)
    W = _rand(g, H, dims["d_h"], dims["d_c"], dtype=dtype, scale=dims["d_c"] ** -0.5)
    pos = torch.randint(0, 1 << 20, (B,), generator=g, dtype=torch.int32).cuda()
    d = abi.make_dims(B=B, H=H, max_pages_per_seq=1, num_pages=1, dtype=dtype, **dims)
    out = torch.empty(B, H, dims["d_c"] + dims["d_r"], dtype=TORCH[dtype], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    abi.absorb_query(d, q, r, pos, W, out, ws)
    abi.check_status(ws)
    want, size = ref.absorb(_np(q), _np(r), pos.cpu().numpy(), _np(W), (dims["d_h"] + dims["d_r"]) ** -0.5)
    tol = (2 * dims["d_h"] + 8) * U32 * size + (U16 * np.abs(want) * (1 + U16) if dtype == "bf16" else 0)
    assert (np.abs(_np(out) - want) <= tol).all()


# ---------------------------------------------------------------------------
# attention weights
# ---------------------------------------------------------------------------
class Weights:
    def __init__(self, dtype, lens, H, nb, dims, seed=0, kernel="auto", scale=2.0):
        g = torch.Generator().manual_seed(seed)
        B, self.nb = len(lens), nb
        self.maxp = max(1, -(-max(lens) // 64)) + 1
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.table, total = _pages(g, lens, self.maxp)
        self.lat = _pool(g, lens, self.table, total, dims["d_c"], dtype)
        self.rope = _pool(g, lens, self.table, total, dims["d_r"], dtype)
        q_scale = scale * ref.LOG2E * (dims["d_c"] / nb + dims["d_r"]) ** -0.5
        self.q = _rand(g, B, H, dims["d_c"] + dims["d_r"], dtype=dtype, scale=q_scale)
        self.dims = abi.make_dims(B=B, H=H, n_branch=nb, max_pages_per_seq=self.maxp, num_pages=total, dtype=dtype,
                                  kernel=kernel, **dims)
        self.lse = self.true_lse()
        self.before = torch.rand(B, self.maxp * 64, generator=g).cuda()
        self.out = torch.full_like(self.before, float("nan"))
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def true_lse(self):
        B, H = self.q.shape[:2]
        lse = np.full((B, self.nb, H), -np.inf)
        d_c = self.lat.shape[-1]
        q, lat, rope = _np(self.q), _np(self.lat), _np(self.rope)
        for b, n in enumerate(self.lens.tolist()):
            c, k = ref.cached(lat, self.table[b].cpu().numpy(), n), ref.cached(rope, self.table[b].cpu().numpy(), n)
            for r in range(self.nb):
                cols = slice(r * d_c // self.nb, (r + 1) * d_c // self.nb)
                if n:
                    s = c[:, cols] @ q[b][:, cols].T + k @ q[b][:, d_c:].T
                    lse[b, r] = np.log2(np.exp2(s - s.max()).sum(0)) + s.max()
        return torch.from_numpy(lse).float().cuda()

    def call(self, before=True, out=None, stream=None):
        abi.attention_weights(self.dims, self.q, self.lse, self.lat, self.rope, self.table, self.lens,
                              self.before if before else None, self.out if out is None else out, self.ws,
                              stream=stream)

    def check(self, before=True):
        abi.check_status(self.ws)
        got, K = _np(self.out), self.lat.shape[-1] // self.nb + self.rope.shape[-1]
        heads = self.nb * self.q.shape[1]
        want = ref.weights(_np(self.q), _np(self.lse), _np(self.lat), _np(self.rope), self.table.cpu().numpy(),
                           self.lens.tolist(), self.nb)
        for b, (p, size) in enumerate(want):
            n = len(p)
            w0 = _np(self.before)[b, :n] if before else 0.0
            # exponents off by 2 K u32 size (and one rounding of the difference): 2^x moves by ln 2 of that
            tol = 2 * (2 * K + 2) * U32 * size + (heads + 16) * U32 * p + U32 * np.abs(p + w0)
            assert (np.abs(got[b, :n] - (w0 + p)) <= tol).all()
            assert np.isnan(got[b, n:]).all(), "weights behind the sequence were written"


WEIGHT_SHAPES = [("f32", TINY, 8, 1), ("f32", TINY, 5, 2), ("bf16", TINY, 3, 1), ("bf16", FULL, 1, 1),
                 ("bf16", FULL, 20, 1), ("bf16", FULL, 32, 1), ("bf16", FULL, 100, 2), ("bf16", FULL, 128, 4),
                 ("bf16", FULL, 128, 1), ("bf16", FULL, 17, 8), ("bf16", dict(FULL, d_r=32), 9, 1),
                 ("bf16", FULL, 130, 1), ("f32", FULL, 4, 4), ("bf16", dict(FULL, d_c=128), 64, 1)]


@pytest.mark.parametrize("dtype,dims,H,nb", WEIGHT_SHAPES)
def test_weights_ragged(dtype, dims, H, nb):
    x = Weights(dtype, (0, 1, 63, 64, 65, 127, 128, 129, 700), H, nb, dims)
    x.call()
    x.check()


@pytest.mark.parametrize("dtype,dims,H,nb", [("bf16", FULL, 32, 1), ("bf16", FULL, 128, 4), ("f32", TINY, 8, 1)])
def test_weights_one_sequence_many_workers(dtype, dims, H, nb):
    x = Weights(dtype, (20001,), H, nb, dims, seed=1)
    x.call(before=False)
    x.check(before=False)


@pytest.mark.parametrize("dtype,dims,H,nb", [("f32", FULL, 3, 2), ("bf16", dict(TINY, d_r=62), 9, 1)])
def test_weights_more_pages_than_workers(dtype, dims, H, nb):
    x = Weights(dtype, (20001, 0, 3000, 77), H, nb, dims, seed=7)
    x.call()
    x.check()


def test_weights_many_sequences_per_worker():
    rng = np.random.default_rng(3)
    x = Weights("bf16", [int(n) for n in rng.integers(0, 300, 400)], 16, 2, FULL, seed=2)
    x.call()
    x.check()


def test_weights_in_place_and_repeatable():
    x = Weights("bf16", (500, 3, 90), 24, 1, FULL, seed=4)
    x.call()
    first, acc = x.out.clone(), x.before.clone()
    x.out.fill_(float("nan"))
    x.call()
    assert torch.equal(first.view(torch.int32), x.out.view(torch.int32))
    x.call(out=acc)
    abi.attention_weights(x.dims, x.q, x.lse, x.lat, x.rope, x.table, x.lens, x.before, x.before, x.ws)
    for b, n in enumerate((500, 3, 90)):
        assert torch.equal(x.before[b, :n], first[b, :n]) and torch.equal(acc[b, :n], first[b, :n])
    abi.check_status(x.ws)


def test_weights_heads_without_a_sum_and_bad_inputs():
    x = Weights("bf16", (200, 70), 12, 1, FULL, seed=5)
    x.lse[0, 0, 3] = float("-inf")
    x.call()
    x.check()
    x.table[1, 1] = -7
    x.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(x.ws)
    x.table[1, 1] = 0
    x.lens[1] = x.maxp * 64 + 1
    x.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(x.ws)


def test_weights_captured():
    x = Weights("bf16", (300, 1000), 32, 1, FULL, seed=6)
    graph = torch.cuda.CUDAGraph()
    x.call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.call()
    x.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    x.check()


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
class Evict:
    def __init__(self, dtype, lens, pages, recent, dims=FULL, seed=0, levels=None, maxp=None):
        g = torch.Generator().manual_seed(seed)
        B, self.recent = len(lens), recent
        self.lens_l, self.pages_l = list(lens), list(pages)
        self.maxp = maxp or max(1, -(-max(lens) // 64)) + 1
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.table, total = _pages(g, lens, self.maxp)
        self.lat = _pool(g, lens, self.table, total, dims["d_c"], dtype)
        self.rope = _pool(g, lens, self.table, total, dims["d_r"], dtype)
        w = torch.rand(B, self.maxp * 64, generator=g)
        self.w = ((w * levels).floor() / levels if levels else w).cuda()
        self.pages = torch.tensor(pages, dtype=torch.int32).cuda()
        self.dims = abi.make_dims(B=B, H=1, max_pages_per_seq=self.maxp, num_pages=total, dtype=dtype, **dims)
        self.ws = torch.zeros(abi.evict_workspace_bytes(self.dims), dtype=torch.uint8, device="cuda")
        self.w_out = torch.full_like(self.w, float("nan"))
        self.table_out, self.lens_out = torch.zeros_like(self.table), torch.zeros_like(self.lens)

    def call(self, stream=None):
        abi.latent_evict(self.dims, self.recent, self.pages, self.w, self.table, self.lens, self.lat, self.rope,
                         self.w_out, self.table_out, self.lens_out, self.ws, stream=stream)

    def expected(self):
        lat, rope = self.lat.clone(), self.rope.clone()
        rows, tables, lens = [], [], []
        table = self.table.cpu().numpy()
        for b, (moves, w, row, n) in enumerate(ref.evict(self.w.cpu().numpy(), table, self.lens_l, self.pages_l,
                                                         self.recent)):
            for s, t in moves:
                for pool, old in ((lat, self.lat), (rope, self.rope)):
                    pool[table[b, t // 64], t % 64] = old[table[b, s // 64], s % 64]
            rows.append(w), tables.append(row), lens.append(n)
        return lat, rope, np.stack(rows), np.stack(tables), lens

    def check(self, want):
        abi.check_status(self.ws)
        lat, rope, w, table, lens = want
        it = torch.int16 if self.lat.dtype == torch.bfloat16 else torch.int32
        assert self.lens_out.tolist() == lens
        np.testing.assert_array_equal(self.table_out.cpu().numpy(), table)
        np.testing.assert_array_equal(self.w_out.cpu().numpy(), w)
        assert torch.equal(self.lat.view(it), lat.view(it)) and torch.equal(self.rope.view(it), rope.view(it))


@pytest.mark.parametrize("dtype,dims", [("f32", TINY), ("bf16", FULL), ("bf16", dict(FULL, d_r=6)),
                                        ("f32", dict(FULL, d_c=96, d_r=2))])
@pytest.mark.parametrize("lens,pages,recent", [
    ((256,), (1,), 32), ((0, 1, 64, 65, 200, 1000), (0, 0, 1, 1, 2, 13), 0), ((500, 700), (0, 10), 60),
    ((128, 640, 333), (2, 9, 5), 0), ((4000, 64, 5000), (31, 0, 70), 200)])
def test_evict(dtype, dims, lens, pages, recent):
    x = Evict(dtype, lens, pages, recent, dims)
    want = x.expected()
    x.call()
    x.check(want)


def test_evict_many_sequences():
    """Warps whose rows lie in several sequences, some of which lose nothing or move nothing."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(0, 700, 500)]
    x = Evict("bf16", lens, [int(rng.integers(0, max(1, n // 64 + 1))) for n in lens], 0,
              dict(d_h=32, d_r=8, d_v=32, d_c=32), seed=8, maxp=70)
    want = x.expected()
    x.call()
    x.check(want)


@pytest.mark.parametrize("levels", [1, 3, 1000])
def test_evict_equal_weights(levels):
    x = Evict("bf16", (3000, 900, 129), (20, 7, 1), 10, levels=levels, seed=1)
    want = x.expected()
    x.call()
    x.check(want)


def test_evict_odd_weights():
    """NaN, infinities, negative numbers, both zeros, subnormals."""
    x = Evict("bf16", (700, 640), (5, 9), 20, seed=2)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf"), -1.0, -0.0, 0.0, 1e-42, -1e-42], device="cuda")
    pick = torch.randint(0, 16, x.w.shape, generator=torch.Generator().manual_seed(3)).cuda()
    x.w = torch.where(pick < 8, odd[pick.clamp_max(7)], x.w)
    want = x.expected()
    x.call()
    x.check(want)


def test_evict_long_sequence_rereads_its_weights():
    """Longer than what the kernel keeps in shared memory; the cache is narrow, so that it stays small."""
    x = Evict("f32", (200000, 131072, 131073), (1000, 2000, 1024), 77, dict(d_h=32, d_r=2, d_v=32, d_c=32), seed=3,
              levels=50)
    want = x.expected()
    x.call()
    x.check(want)


def test_evict_again_and_captured():
    x = Evict("bf16", (900, 2000), (6, 20), 64, seed=4)
    want = x.expected()
    x.call()
    x.check(want)
    x.call()  # the same call again moves the same tokens
    x.check(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.call()
    x.w_out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    x.check(want)


@pytest.mark.parametrize("pages", [-1, 9, 1 << 25])
def test_evict_more_than_there_is_is_reported(pages):
    x = Evict("bf16", (600, 500), (4, 5), 30, seed=5)
    x.pages_l[0] = 0
    want = x.expected()
    x.pages[0] = pages
    x.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(x.ws)
    x.check(want)


def test_evict_does_not_write_shared_or_missing_pages():
    x = Evict("bf16", (640, 640), (4, 0), 0, seed=6)
    x.table[1, 3:8] = x.table[0, 3:8]  # a part of the second sequence lies in the first one's pages
    x.table[0, 8] = -5
    before = x.lat.clone()
    x.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(x.ws)
    kept = x.table[1, :10].long()
    assert torch.equal(x.lat[kept].view(torch.int16), before[kept].view(torch.int16))
    assert x.lens_out.tolist() == [640 - 256, 640]


# ---------------------------------------------------------------------------
# together, as a serving loop uses them
# ---------------------------------------------------------------------------
def test_prompt_decode_evict_append_decode():
    """A prompt, its first token with the weights it gives, an eviction, the next token: each step against the
    64-bit forms, the last one over exactly the tokens that were kept."""
    g = torch.Generator().manual_seed(9)
    lens, H, D = [400, 130], 16, 256
    w = FULL
    B, T, maxp = 2, sum(lens), 8
    c, kr = _rand(g, T, w["d_c"], dtype="bf16"), _rand(g, T, w["d_r"], dtype="bf16")
    W_UK = _rand(g, H, w["d_h"], w["d_c"], dtype="bf16", scale=w["d_c"] ** -0.5)
    W_UV = _rand(g, H, w["d_c"], w["d_v"], dtype="bf16", scale=w["d_c"] ** -0.5)
    seq = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32).cuda()
    pos = torch.tensor([t for n in lens for t in range(n)], dtype=torch.int32).cuda()
    table, total = _pages(g, [maxp * 64] * B, maxp)
    d = abi.make_dims(B=B, H=H, max_pages_per_seq=maxp, num_pages=total, **w)
    lat = torch.full((total, 64, w["d_c"]), float("nan"), dtype=torch.bfloat16, device="cuda")
    rope = torch.full((total, 64, w["d_r"]), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(abi.workspace_bytes(d), dtype=torch.uint8, device="cuda")
    abi.latent_store(d, T, c, kr, seq, pos, table, lat, rope, ws)
    # the prompt
    cu = torch.tensor([0, lens[0], T], dtype=torch.int32).cuda()
    q, qr = _rand(g, T, H, w["d_h"], dtype="bf16"), _rand(g, T, H, w["d_r"], dtype="bf16")
    k = torch.einsum("tc,hdc->thd", c.float(), W_UK.float()).bfloat16()
    v = torch.einsum("tc,hcd->thd", c.float(), W_UV.float()).bfloat16()
    out = torch.empty(T, H, w["d_v"], dtype=torch.bfloat16, device="cuda")
    pws = torch.zeros(abi.prompt_workspace_bytes(d, T, T, H), dtype=torch.uint8, device="cuda")
    abi.mla_prompt(d, q, qr, cu, k, v, cu, rope, table, out, pws)
    # the prompt's last rows are the decode of the same tokens, in the absorbed form (bf16 roundings on both sides)
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    last = (cu[1:] - 1).long()
    dec = torch.empty(B, H, w["d_v"], dtype=torch.bfloat16, device="cuda")
    args = (q[last].contiguous(), qr[last].contiguous(), seq_lens - 1)
    abi.mla_decode(d, *args, W_UK, W_UV, lat, rope, table, seq_lens, dec, ws)
    scale = (w["d_h"] + w["d_r"]) ** -0.5
    exact = _decode64(args, W_UK, W_UV, lat, rope, table, lens, scale)
    for got in (dec, out[last]):
        assert np.abs(_np(got) - exact).max() <= 1e-2 * np.abs(exact).max() + 1e-3
    # what each token was worth, from the same step's log-sum-exp
    o = torch.empty(B, H, w["d_c"], device="cuda")
    lse = torch.empty(B, 1, H, device="cuda")
    abi.attend_partial(d, *args, W_UK, lat, rope, table, seq_lens, o, lse, ws)
    q_abs = torch.empty(B, H, w["d_c"] + w["d_r"], dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros(B, maxp * 64, device="cuda")
    abi.absorb_query(d, *args, W_UK, q_abs, ws)
    abi.attention_weights(d, q_abs, lse, lat, rope, table, seq_lens, weights, weights, ws)
    # a head's weights add up to one: both sides take the same rounded query; the scores are the tolerance's
    # 2 K u32 sum|q||c|, about 1e-4 here at most
    np.testing.assert_allclose(_np(weights).sum(1), H, rtol=1e-3)
    # evict two pages of the long sequence, one of the short; then the next token
    ews = torch.zeros(abi.evict_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    pages = torch.tensor([2, 1], dtype=torch.int32).cuda()
    w2, table2, lens2 = torch.empty_like(weights), torch.empty_like(table), torch.empty_like(seq_lens)
    kept_lat, kept_rope = lat.clone(), rope.clone()
    abi.latent_evict(d, 16, pages, weights, table, seq_lens, lat, rope, w2, table2, lens2, ews)
    h, W_D, W_R = _rand(g, B, D, dtype="bf16"), _rand(g, D, w["d_c"], dtype="bf16", scale=D ** -0.5), \
        _rand(g, D, w["d_r"], dtype="bf16", scale=D ** -0.5)
    aws = torch.zeros(abi.append_workspace_bytes(d, D), dtype=torch.uint8, device="cuda")
    abi.latent_append(d, D, h, W_D, W_R, seq_lens, table, lat, rope, aws)  # by position: the table from before
    nxt = (_rand(g, B, H, w["d_h"], dtype="bf16"), _rand(g, B, H, w["d_r"], dtype="bf16"), seq_lens)
    abi.mla_decode(d, *nxt, W_UK, W_UV, lat, rope, table2, lens2 + 1, dec, ws)
    for x in (ws, pws, ews, aws):
        abi.check_status(x)
    tab, wn = table.cpu().numpy(), weights.cpu().numpy()
    for b, (moves, _, _, n) in enumerate(ref.evict(wn, tab, lens, [2, 1], 16)):
        keep = sorted(({t for t in range(lens[b])} - {t for t in range(pages[b] * 64)} - {t for _, t in moves})
                      | {s for s, _ in moves}) if moves else list(range(int(pages[b]) * 64, lens[b]))
        assert len(keep) == n
        slot = lambda pool, t: _np(pool[tab[b, t // 64], t % 64])  # noqa: E731
        cs = np.stack([slot(kept_lat, t) for t in keep] + [slot(lat, lens[b])])
        ks = np.stack([slot(kept_rope, t) for t in keep] + [slot(rope, lens[b])])
        want = _rows64([x[b:b + 1] for x in nxt], W_UK, W_UV, cs, ks, scale)
        assert np.abs(_np(dec[b]) - want).max() <= 1e-2 * np.abs(want).max() + 1e-3


def _rows64(args, W_UK, W_UV, c, k, scale):
    q, qr, pos = (_np(x) for x in args)
    rot = ref.rope(qr, pos[:, None])
    out = np.zeros((q.shape[1], W_UV.shape[2]))
    for h in range(q.shape[1]):
        x = scale * (c @ (q[0, h] @ _np(W_UK[h])) + k @ rot[0, h])
        p = np.exp(x - x.max())
        out[h] = (p / p.sum()) @ c @ _np(W_UV[h])
    return out


def _decode64(args, W_UK, W_UV, lat, rope, table, lens, scale):
    rows = []
    for b, n in enumerate(lens):
        row = table[b].cpu().numpy()
        rows.append(_rows64([x[b:b + 1] for x in args], W_UK, W_UV, ref.cached(_np(lat), row, n),
                            ref.cached(_np(rope), row, n), scale))
    return np.stack(rows)
