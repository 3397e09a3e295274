"""More of the operators around the decode step on the GPU: values that are
not finite where the mask hides them, many work items per CTA, groups of heads,
peaked scores, sequences that overlap.

The bounds are those of test_gpu_serving.py, the 64-bit form is torch's own
matrix product in float64, one (sequence, head) at a time.
"""
import math

import pytest
import torch

from mlra_latent_kv_b200 import abi
from test_gpu_serving import FULL, TINY, U16, U32, Evict, Prompt, Weights

pytestmark = pytest.mark.gpu

LOG2E = math.log2(math.e)


def _prompt(dtype, q_lens, k_lens, H, kv, **kw):
    return Prompt(dtype, q_lens, k_lens, H, kv, dims=FULL if dtype == "bf16" else TINY, **kw)


def _bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


def _rotated(x, pos):
    d = x.shape[-1]
    ang = pos.double()[:, None] * 10000.0 ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    c, s, out = ang.cos(), ang.sin(), torch.empty_like(x)
    out[:, 0::2] = x[:, 0::2] * c - x[:, 1::2] * s
    out[:, 1::2] = x[:, 0::2] * s + x[:, 1::2] * c
    return out


def _exact(p, b, h, v):
    """(rows, out, its bound, lse, its bound) of one sequence and head in 64 bits, `v` in place of the values."""
    q0, q1, k0, k1 = (int(cu[b + i]) for cu in (p.cu_q, p.cu_k) for i in (0, 1))
    lq, lk, g = q1 - q0, k1 - k0, h // (p.H // p.kv)
    pos = torch.arange(lq, device="cuda") + lk - lq
    pages = p.table[b, :-(-lk // 64)].long()
    rope = p.rope_cache[pages].reshape(-1, p.w["d_r"])[:lk].double()
    qn, kn, val = p.q_nope[q0:q1, h].double(), p.k_nope[k0:k1, g].double(), v[k0:k1, g].double()
    qr = _rotated(p.q_rope[q0:q1, h].double(), pos)
    seen = torch.arange(lk, device="cuda")[None] <= pos[:, None]
    x = (p.scale * (qn @ kn.T + qr @ rope.T)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, 1)
    w = torch.where(seen, (x - lse[:, None]).exp(), 0)
    out, spread = w @ val, w @ val.abs()
    rot = p.scale * qr.abs() @ rope.abs().T
    dot = (rot + p.scale * qn.abs() @ kn.abs().T).masked_fill(~seen, 0).amax(1) if lk else x.sum(1)
    rot = rot.masked_fill(~seen, 0).amax(1) if lk else dot
    off = 2 * (p.w["d_h"] + p.w["d_r"] + 4) * U32 * dot
    if p.dtype == "bf16":
        off = off + U16 * rot
    tol = (torch.expm1(2 * off)[:, None] + (2 * lk + 16) * U32) * spread + 1e-30
    if p.dtype == "bf16":
        tol = tol * (1 + U16) + U16 * spread * (1 + U16) + U16 * out.abs()
    lse_tol = off * LOG2E + (lk + 16) * U32 * LOG2E + 4 * U32 * (lse * LOG2E).abs().nan_to_num(posinf=0)
    return slice(q0, q1), out, tol, lse * LOG2E, lse_tol


def _check(p, heads=None, v=None, skip=None):
    """Compares the outputs of `heads` (all of them) with the 64-bit form; `skip`: outputs that are looked at elsewhere.
    Returns the median of bound / |output|."""
    abi.check_status(p.ws)
    ratio = []
    for b in range(len(p.cu_q) - 1):
        for h in range(p.H) if heads is None else heads:
            rows, out, tol, lse, lse_tol = _exact(p, b, h, p.v if v is None else v)
            err = (p.out[rows, h].double() - out).abs()
            ok = err <= tol
            if skip is not None:
                ok |= skip[rows, h]
            assert ok.all(), f"sequence {b}, head {h}: {int((~ok).sum())} outputs, {(err / tol).max():.2f} of the bound"
            got, none = p.lse[rows, h].double(), lse.isneginf()
            assert got[none].isneginf().all() and ((got - lse).abs() <= lse_tol)[~none].all()
            ratio.append((tol / out.abs())[out != 0].flatten())
    assert p.out[int(p.cu_q[-1]):].isnan().all() and p.lse[int(p.cu_q[-1]):].isnan().all()
    return torch.cat(ratio).median().item()


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,H,kv", [("f32", 4, 4), ("f32", 6, 2), ("bf16", 4, 4), ("bf16", 16, 2), ("bf16", 128, 1)])
def test_prompt_values_of_later_tokens_do_not_reach_a_query(dtype, H, kv, bad):
    """A value that is not finite is the output of the queries that see it, in its own column; nothing else changes."""
    q_lens, k_lens = (300, 5, 140), (300, 700, 200)
    p = _prompt(dtype, q_lens, k_lens, H, kv, seed=20)
    clean, hit = p.v.clone(), torch.zeros_like(p.out, dtype=torch.bool)
    # sequence, kv head, key, column
    for b, g, j, c in ((0, 0, 211, 3), (0, kv - 1, 90, 17), (1, 0, 698, 0), (2, kv - 1, 199, 31), (2, 0, 61, 8)):
        p.v[int(p.cu_k[b]) + j, g, c] = bad
        first = max(0, j - (k_lens[b] - q_lens[b]))  # the first query that sees key j
        hit[int(p.cu_q[b]) + first:int(p.cu_q[b + 1]), g * (H // kv):(g + 1) * (H // kv), c] = True
    p.call()
    _check(p, v=clean, skip=hit)
    torch.testing.assert_close(p.out[hit].float(), torch.full_like(p.out[hit].float(), bad), equal_nan=True)


@pytest.mark.parametrize("dtype,H,kv", [("f32", 4, 2), ("bf16", 4, 4), ("bf16", 16, 2)])
def test_prompt_tokens_whose_values_are_all_nan(dtype, H, kv):
    """The tokens behind the first of them, too: a row that is NaN as it is, and rows before it with a second one."""
    p = _prompt(dtype, (400, 130), (400, 390), H, kv, seed=22)
    clean, hit = p.v.clone(), torch.zeros_like(p.out, dtype=torch.bool)
    p.v[[150, 160, 399, 400 + 300]] = float("nan")
    p.v[140, 0, 5] = float("inf")
    hit[150:400], hit[400 + 40:400 + 130], hit[140:150, :H // kv, 5] = True, True, True  # 300 - (390 - 130) = 40
    p.call()
    _check(p, v=clean, skip=hit)
    assert p.out[150:400].isnan().all() and p.out[440:530].isnan().all() and p.out[140:150, :H // kv, 5].isposinf().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_keys_of_later_tokens_do_not_reach_a_query(dtype):
    p = _prompt(dtype, (200, 90), (260, 90), 4, 2, seed=21)
    p.call()
    want, want_lse = p.out.clone(), p.lse.clone()
    p.k_nope[230] = float("nan")  # seen from query 170 of the first sequence on
    p.k_nope[260 + 64] = float("inf")
    p.rope_cache[p.table[1, 1].long(), 20] = float("nan")  # key 84 of the second
    p.call()
    for rows in (slice(0, 170), slice(200, 264)):
        assert torch.equal(_bits(p.out[rows]), _bits(want[rows])) and torch.equal(p.lse[rows], want_lse[rows])
    assert p.out[170:200].isnan().all() and p.out[284:290].isnan().all()


# ---------------------------------------------------------------------------
# sequences that overlap
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_overlapping_sequences_stay_in_the_workspace(dtype):
    """41 times the same rows, with a descending pair of offsets between them: more tiles than the lists have room for."""
    T, B = 1024, 81
    p = _prompt(dtype, (T,) + (0,) * (B - 1), (T,) + (0,) * (B - 1), 2, 2, seed=23)
    assert (B + 1) // 2 * T // 256 > (p.out.shape[0] + 255) // 256 + B
    for cu in (p.cu_q, p.cu_k):
        cu[:] = torch.tensor([T * (i % 2) for i in range(B + 1)], dtype=torch.int32)
    p.table[:] = p.table[:1].clone()
    size, guard = p.ws.numel(), 1 << 16
    whole = torch.full((size + guard,), 0x5a, dtype=torch.uint8, device="cuda")
    whole[:256] = 0
    p.ws = whole[:size]
    p.call()
    with pytest.raises(abi.MlraError):
        abi.check_status(p.ws)
    assert (whole[size:] == 0x5a).all()
    assert p.out[T:].isnan().all() and p.lse[T:].isnan().all()
    if dtype == "bf16":  # the plan is not made: no row is written, and no item listed
        assert p.out.isnan().all() and p.lse.isnan().all()
        assert (whole[512:512 + 8 * (T // 256 + B)] == 0x5a).all()


# ---------------------------------------------------------------------------
# peaked scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,kernel", [("f32", "auto"), ("bf16", "auto"), ("bf16", "simt")])
def test_prompt_peaked_scores(dtype, kernel):
    """Scores of a standard deviation of 24 (fp32: 49) without a rotary part, whose rounding would be most of the bound:
    the running maximum jumps by far more than the kernel puts up with, and the bound stays near the output's rounding."""
    p = _prompt(dtype, (150, 300), (150, 700), 4, 4, scale=30.0 if dtype == "bf16" else 60.0, seed=24, kernel=kernel)
    p.q_rope[:] = 0
    p.call()
    assert _check(p) < 0.05


def test_prompt_scores_that_rise():
    """By 0.14 a key: the maximum moves by 18 in every step of 128 keys, and only a row's last keys count."""
    p = _prompt("bf16", (500,), (900,), 2, 1, scale=0.1, seed=25)
    p.q_rope[:] = 0
    p.q_nope[:, :, 0] = 1.0
    p.k_nope[:900, :, 0] = (2.0 * torch.arange(900, device="cuda")).to(torch.bfloat16)[:, None]
    p.call()
    assert _check(p) < 0.05


# ---------------------------------------------------------------------------
# more work items than CTAs
# ---------------------------------------------------------------------------
def _items(p):
    """Pairs of 128-row tiles of the tcgen05 kernel."""
    group = p.H // p.kv
    pack = min(128, group & -group)
    pairs = sum(-(-int(n) * pack // 256) for n in p.cu_q[1:] - p.cu_q[:-1])
    return pairs * (p.H // pack)


def _twice(p):
    p.call()
    out, lse = p.out.clone(), p.lse.clone()
    p.out.fill_(float("nan"))
    p.lse.fill_(float("nan"))
    p.call()
    assert torch.equal(_bits(out), _bits(p.out)) and torch.equal(_bits(lse), _bits(p.lse))


# single tokens, key lengths around the tiles' ends, contexts, more queries than keys (whose first tiles have no key),
# sequences without queries or keys: what one item leaves behind meets every kind of next one
MIXED_Q = (1, 700, 64, 257, 129, 5, 0, 300, 128, 3, 513, 40, 256, 90, 1, 640)
MIXED_K = (1, 700, 500, 257, 130, 900, 70, 10, 128, 0, 800, 1300, 255, 91, 2000, 300)


@pytest.mark.parametrize("H,kv", [(32, 32), (48, 16), (96, 48)])
def test_prompt_several_items_a_cta(H, kv):
    p = _prompt("bf16", MIXED_Q, MIXED_K, H, kv, seed=26)
    assert _items(p) > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    _twice(p)
    _check(p)


def test_prompt_several_items_a_cta_of_packed_heads():
    p = _prompt("bf16", MIXED_Q * 3, MIXED_K * 3, 64, 4, seed=27)
    assert _items(p) > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    _twice(p)
    _check(p, heads=(0, 17, 38, 63))


def test_prompt_many_items_with_values_that_are_not_finite():
    """Items to be taken again between others that are not, several of a CTA."""
    H, kv = 48, 24
    p = _prompt("bf16", MIXED_Q * 2, MIXED_K * 2, H, kv, seed=28)
    clean, hit = p.v.clone(), torch.zeros_like(p.out, dtype=torch.bool)
    for b in range(0, len(MIXED_Q) * 2, 3):
        q0, q1, k0, k1 = (int(cu[b + i]) for cu in (p.cu_q, p.cu_k) for i in (0, 1))
        for n, g in enumerate(range(b % 2, kv, 2)):
            j = (k1 - k0) * (n + 1) // kv  # the keys of a prompt's first half and more
            if j < k1 - k0:
                p.v[k0 + j, g, b] = float("inf")
                hit[q0 + max(0, j - (k1 - k0 - (q1 - q0))):q1, 2 * g:2 * g + 2, b] = True
    _twice(p)
    _check(p, v=clean, skip=hit)
    assert p.out[hit].isposinf().all()


@pytest.mark.parametrize("H,kv", [(128, 128), (128, 64)])
def test_prompt_groups_of_heads(H, kv):
    """More K and V than L2 holds: the heads are taken in groups, the last of them smaller (128 kv heads: 43 + 43 + 42)."""
    p = _prompt("bf16", (300, 2), (4100, 200), H, kv, seed=29)
    units = H // (H // kv)
    group = (112 << 20) // (p.k_nope.shape[0] * 512 * kv // units)
    groups = -(-units // group)
    assert groups > 1 and (kv < 128 or units % groups)
    assert _items(p) > torch.cuda.get_device_properties(0).multi_processor_count
    _twice(p)
    _check(p, heads=(0, 1, 41, 42, 43, 44, 85, 86, 87, 126, 127))


def test_prompt_two_calls_at_once():
    """Two batches on two streams, a workspace each: the same bits as one after the other."""
    a, b = (_prompt("bf16", MIXED_Q, MIXED_K, 24, 24, seed=30 + i) for i in range(2))
    a.call()
    b.call()
    want = [x.clone() for x in (a.out, b.out, a.lse, b.lse)]
    for x in (a, b):
        x.out.fill_(float("nan"))
        x.lse.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, s in zip((a, b), streams):
            p.call(stream=s)
    torch.cuda.synchronize()
    for x, y in zip(want, (a.out, b.out, a.lse, b.lse)):
        assert torch.equal(_bits(x), _bits(y))
    abi.check_status(a.ws)
    abi.check_status(b.ws)


# ---------------------------------------------------------------------------
# eviction and weights
# ---------------------------------------------------------------------------
def test_evict_of_a_shared_prefix_reads_it_for_each_sequence():
    """Three sequences begin with the same four pages; two of them give exactly these up, the third keeps them."""
    x = Evict("bf16", (1000, 700, 500), (4, 4, 0), 20, seed=40)
    x.table[1:, :4] = x.table[:1, :4].clone()
    x.lat.nan_to_num_(0.5), x.rope.nan_to_num_(0.5)  # the pages that nobody names any more
    want = x.expected()
    prefix = x.table[0, :4].long()
    before = x.lat[prefix].clone()
    x.call()
    x.check(want)
    assert torch.equal(_bits(x.lat[prefix]), _bits(before))


def test_weights_and_evict_on_another_stream():
    w, e = Weights("bf16", (3000, 77), 32, 1, FULL, seed=41), Evict("bf16", (900, 2000), (6, 20), 64, seed=42)
    want = e.expected()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w.call(stream=side)
    e.call(stream=side)
    with torch.cuda.stream(side):  # and on the stream that is current
        e.call()
        w.call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    w.check()
    e.check(want)
