"""The operators of the prompt and of cache eviction, as measured cases.

Four operators of a serving loop over the paged latent cache:

  prompt    causal attention of whole prompts (packed, ragged, with or without
            an earlier context, grouped heads) in the unabsorbed form, the
            decoupled RoPE keys read from the paged cache
  absorb    the decode query folded through W_UK and rotated: what the scores
            against the cached latent are taken with
  weights   each cached token's attention weight, summed over heads and
            branches and added to what it has gathered so far
  evict     whole pages freed per sequence: the tokens with the least weight
            go, the tokens to keep move into their slots

``run`` computes a case in elementary torch operations, or (``own``) through
the library's entry points.  ``exact`` computes it again in 64 bits.
"""
import math
import random

import torch

own = False

PAGE = 64
LOG2E = 1.4426950408889634
ROPE_BASE = 10000.0
# widths of the library's own configurations: (d_h, d_r, d_v, d_c)
WIDTHS = {"full": (128, 64, 128, 512), "tiny": (32, 16, 32, 64)}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tiny fp32 configuration's prompt: one short sequence, where latency counts
        {"name": "prompt tiny fp32", "op": "prompt", "dtype": "f32", "widths": "tiny", "H": 8, "kv_heads": 8, "B": 1,
         "lo": 256, "hi": 256, "ctx": 0, "lens": 1},
        # one full prompt of the 128-head configuration: the tensor cores' case
        {"name": "prompt 128 heads", "op": "prompt", "dtype": "bf16", "widths": "full", "H": 128, "kv_heads": 128,
         "B": 1, "lo": 4096, "hi": 4096, "ctx": 0, "lens": 2},
        # a packed batch of prompts of very different lengths, from a single token on
        {"name": "prompt packed ragged", "op": "prompt", "dtype": "bf16", "widths": "full", "H": 32, "kv_heads": 32,
         "B": 16, "lo": 1, "hi": 1900, "ctx": 0, "lens": 3},
        # chunks of prompts whose earlier part is cached already, with grouped heads
        {"name": "prompt chunk grouped", "op": "prompt", "dtype": "bf16", "widths": "full", "H": 32, "kv_heads": 8,
         "B": 4, "lo": 200, "hi": 800, "ctx": 8000, "lens": 4},
        # the query side of a decode step, at the paged and at the 128-head configuration
        {"name": "absorb 32 heads", "op": "absorb", "dtype": "bf16", "widths": "full", "H": 32, "B": 64},
        {"name": "absorb 128 heads", "op": "absorb", "dtype": "bf16", "widths": "full", "H": 128, "B": 32},
        # the weights of the tiny fp32 configuration's cache
        {"name": "weights tiny fp32", "op": "weights", "dtype": "f32", "widths": "tiny", "H": 8, "branches": 1, "B": 1,
         "lo": 256, "hi": 256, "lens": 5},
        # a paged batch of 32 heads over lengths from 1024 to 32768
        {"name": "weights paged 32 heads", "op": "weights", "dtype": "bf16", "widths": "full", "H": 32, "branches": 1,
         "B": 64, "lo": 1024, "hi": 32768, "lens": 6},
        # four branches of 128 heads each
        {"name": "weights four branches", "op": "weights", "dtype": "bf16", "widths": "full", "H": 128, "branches": 4,
         "B": 32, "lo": 16384, "hi": 16384, "lens": 7},
        # one short fp32 sequence that loses a page
        {"name": "evict tiny fp32", "op": "evict", "dtype": "f32", "widths": "tiny", "B": 1, "lo": 256, "hi": 256,
         "recent": 32, "share": 0.3, "lens": 8},
        # a paged batch that is brought to about half its length
        {"name": "evict paged batch", "op": "evict", "dtype": "bf16", "widths": "full", "B": 64, "lo": 1024,
         "hi": 32768, "recent": 128, "share": 0.5, "lens": 9},
        # four long contexts that lose three quarters
        {"name": "evict long contexts", "op": "evict", "dtype": "bf16", "widths": "full", "B": 4, "lo": 131072,
         "hi": 131072, "recent": 1000, "share": 0.75, "lens": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "absorb", "weights", "weights", "evict", "evict"])
    tiny = rng.random() < 0.25
    c = {"op": op, "dtype": "f32" if tiny else "bf16", "widths": "tiny" if tiny else "full"}
    if op == "prompt":
        if tiny:
            heads, B = rng.choice([1, 3, 8]), rng.randint(1, 4)
            hi = _log(rng, 1, 500)
            ctx = rng.choice([0, 0, rng.randint(1, 300)])
        else:
            heads, B = rng.choice([8, 16, 24, 32, 64, 128]), _log(rng, 1, 16)
            hi = _log(rng, 1, 4096)
            ctx = rng.choice([0, 0, _log(rng, 1, 8000)])
            while B * heads * hi * (hi + ctx) > 2 ** 30:  # within half of the largest listed case
                B, hi, ctx = max(1, B // 2), max(1, hi * 3 // 4), ctx * 3 // 4
        groups = [g for g in (1, 1, 1, 2, 3, 4, 8) if heads % g == 0]
        return c | {"H": heads, "kv_heads": heads // rng.choice(groups), "B": B, "lo": rng.randint(1, hi), "hi": hi,
                    "ctx": ctx, "lens": rng.randrange(1 << 20)}
    if op == "absorb":
        return c | {"H": rng.choice([8, 20, 32, 64, 128]), "B": _log(rng, 1, 64)}
    if op == "weights":
        if tiny:
            return c | {"H": rng.randint(1, 8), "branches": rng.choice([1, 2]), "B": rng.randint(1, 4),
                        "lo": 1, "hi": _log(rng, 1, 2000), "lens": rng.randrange(1 << 20)}
        H, branches, hi = rng.choice([5, 16, 20, 32, 64, 100, 128]), rng.choice([1, 1, 2, 4]), _log(rng, 64, 60000)
        B = max(1, min(_log(rng, 1, 64), 400000 // hi))
        return c | {"H": H, "branches": branches, "B": B, "lo": rng.randint(1, hi), "hi": hi,
                    "lens": rng.randrange(1 << 20)}
    hi = _log(rng, 100, 2000 if tiny else 100000)
    B = max(1, min(_log(rng, 1, 64), 400000 // hi))
    return c | {"B": B, "lo": rng.randint(1, hi), "hi": hi, "recent": rng.randint(0, min(hi, 300)),
                "share": round(rng.uniform(0.02, 0.95), 2), "lens": rng.randrange(1 << 20)}


def _lens(case):
    """Lengths of the case's sequences: spread over [lo, hi] on a logarithmic scale, the longest among them."""
    rng = random.Random(case["lens"])
    lens = [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[rng.randrange(case["B"])] = case["hi"]
    return lens


def _contexts(case):
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(case["ctx"] // 2, case["ctx"]) for _ in range(case["B"])]


def _evict_pages(case):
    """Pages that each sequence gives up: `share` of it, as far as its recent tokens leave room."""
    return [min(int(n * case["share"]) // PAGE, max(0, n - case["recent"]) // PAGE) for n in _lens(case)]


def _scale(case):
    d_h, d_r, _, _ = WIDTHS[case["widths"]]
    return 1.0 / math.sqrt(d_h + d_r)


def work(case):
    d_h, d_r, d_v, d_c = WIDTHS[case["widths"]]
    e = 4 if case["dtype"] == "f32" else 2
    B, op = case["B"], case["op"]
    if op == "prompt":
        H, kv = case["H"], case["kv_heads"]
        q, ctx = _lens(case), _contexts(case)
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(q, ctx))
        rows = sum(q) * H * (d_h + d_r + d_v)
        keys = (sum(q) + sum(ctx)) * (kv * (d_h + d_v) + d_r)
        return {"bytes": (rows + keys) * e, "flops": 2 * pairs * H * (d_h + d_r + d_v)}
    if op == "absorb":
        H = case["H"]
        return {"bytes": (H * d_h * d_c + B * H * (d_h + d_r) + B * H * (d_c + d_r)) * e + 4 * B,
                "flops": 2 * B * H * d_h * d_c}
    n = _lens(case)
    if op == "weights":
        H, nb = case["H"], case["branches"]
        # the rotary part of a score is the same in every branch
        return {"bytes": sum(n) * ((d_c + d_r) * e + 8) + B * H * ((d_c + d_r) * e + 4 * nb),
                "flops": 2 * sum(n) * H * (d_c + d_r)}
    # evict: of each page that goes, the tokens that stay (their number depends on the weights: the share that is
    # kept) are read and written, the weights are read and written
    moved = sum(PAGE * p * (1 - PAGE * p / max(1, m - case["recent"])) for m, p in zip(n, _evict_pages(case)))
    row = -(-max(n) // PAGE) * PAGE
    return {"bytes": 2 * moved * (d_c + d_r) * e + 4 * sum(n) + 4 * B * row, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _pages(g, lens, spare=3):
    """A pool in which every sequence's pages lie in a random order: (page_table [B, widest], pages in the pool)."""
    counts = [-(-n // PAGE) for n in lens]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _pool(g, lens, table, total, width, dtype):
    """A page pool with random tokens; the slots that no sequence uses hold NaN, as memory nobody wrote may."""
    pool = torch.randn(total, PAGE, width, generator=g, device="cuda", dtype=torch.bfloat16).to(dtype)
    used = torch.zeros(total, PAGE, dtype=torch.bool, device="cuda")
    slot = torch.arange(table.shape[1] * PAGE, device="cuda")
    valid = slot[None, :] < torch.tensor(lens, device="cuda")[:, None]
    used.view(-1)[(table.long().repeat_interleave(PAGE, 1) * PAGE + slot % PAGE)[valid]] = True
    pool[~used] = float("nan")
    return pool


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    d_h, d_r, d_v, d_c = WIDTHS[case["widths"]]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    s = {"case": case, "scale": _scale(case)}
    op, B = case["op"], case["B"]
    if op == "prompt":
        H, kv = case["H"], case["kv_heads"]
        q_lens = _lens(case)
        k_lens = [n + c for n, c in zip(q_lens, _contexts(case))]
        s["cu_q"] = _int([sum(q_lens[:b]) for b in range(B + 1)])
        s["cu_k"] = _int([sum(k_lens[:b]) for b in range(B + 1)])
        # as the projections leave them: query heads of d_h + d_r, key heads of d_h + d_v
        q = _randn(g, sum(q_lens), H, d_h + d_r, dtype=dt)
        kv_up = _randn(g, sum(k_lens), kv, d_h + d_v, dtype=dt)
        s["q_nope"], s["q_rope"] = q[..., :d_h], q[..., d_h:]
        s["k_nope"], s["v"] = kv_up[..., :d_h], kv_up[..., d_h:]
        s["page_table"], total = _pages(g, k_lens)
        s["rope_cache"] = _pool(g, k_lens, s["page_table"], total, d_r, dt)
        s["out"] = torch.zeros(sum(q_lens), H, d_v, dtype=dt, device="cuda")
        s["longest"] = (max(q_lens), max(k_lens))
    elif op == "absorb":
        H = case["H"]
        s["q_nope"], s["q_rope"] = _randn(g, B, H, d_h, dtype=dt), _randn(g, B, H, d_r, dtype=dt)
        s["q_pos"] = torch.randint(0, 131072, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["W_UK"] = _randn(g, H, d_h, d_c, scale=d_c ** -0.5, dtype=dt)
        s["q_abs"] = torch.empty(B, H, d_c + d_r, dtype=dt, device="cuda")
        total = 1
        s["page_table"] = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    else:
        lens = _lens(case)
        s["seq_lens"] = _int(lens)
        s["page_table"], total = _pages(g, lens)
        s["latent_cache"] = _pool(g, lens, s["page_table"], total, d_c, dt)
        s["rope_cache"] = _pool(g, lens, s["page_table"], total, d_r, dt)
        slots = s["page_table"].shape[1] * PAGE
        valid = torch.arange(slots, device="cuda")[None, :] < s["seq_lens"][:, None]
        # weights gathered so far, a few tokens with far more than the others; their mean is one step's share
        heads = case.get("H", 1) * case.get("branches", 1)
        gathered = torch.rand(B, slots, generator=g, device="cuda").clamp_min_(1e-7).log_().square_().mul_(heads / 2)
        s["weights_in"] = torch.where(valid, gathered / s["seq_lens"][:, None], 0.0)
        s["weights"] = torch.zeros_like(s["weights_in"])
        if op == "weights":
            H, nb = case["H"], case["branches"]
            # an absorbed query: logits with a standard deviation of about two
            q = _randn(g, B, H, d_c + d_r)
            q[..., :d_c] *= (d_h / d_c) ** 0.5
            s["q_abs"] = (q * (2 * s["scale"] * LOG2E * nb ** 0.5)).to(dt)
            x = _scores(s).masked_fill_(~valid[:, None, None, :], float("-inf"))
            top = x.amax(-1, keepdim=True)
            s["lse"] = top[..., 0] + x.sub_(top).exp2_().sum(-1).log2()
        else:
            s["evict_pages"] = _int(_evict_pages(case))
            # equal weights are ordinary too: tokens that no query has met yet
            s["weights_in"][torch.rand(B, slots, generator=g, device="cuda") < 0.05] = 0.0
            s["page_table_out"] = torch.empty_like(s["page_table"])
            s["seq_lens_out"] = torch.empty_like(s["seq_lens"])
    if own:
        from mlra_latent_kv_b200 import abi
        s["dims"] = abi.make_dims(B=B, H=case.get("H", 1), d_h=d_h, d_v=d_v, d_c=d_c, d_r=d_r,
                                  max_pages_per_seq=s["page_table"].shape[1], num_pages=total,
                                  n_branch=case.get("branches", 1), dtype=case["dtype"])
        n = abi.prompt_workspace_bytes(s["dims"], s["q_nope"].shape[0], s["k_nope"].shape[0], case["kv_heads"]) \
            if op == "prompt" else abi.evict_workspace_bytes(s["dims"]) if op == "evict" else 256
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _RUN_OWN[op](s)
    return _RUN_PLAIN[op](s)


def _own_prompt(s):
    from mlra_latent_kv_b200 import abi
    abi.mla_prompt(s["dims"], s["q_nope"], s["q_rope"], s["cu_q"], s["k_nope"], s["v"], s["cu_k"], s["rope_cache"],
                   s["page_table"], s["out"], s["workspace"])
    return s["out"]


def _own_absorb(s):
    from mlra_latent_kv_b200 import abi
    abi.absorb_query(s["dims"], s["q_nope"], s["q_rope"], s["q_pos"], s["W_UK"], s["q_abs"], s["workspace"])
    return s["q_abs"]


def _own_weights(s):
    from mlra_latent_kv_b200 import abi
    abi.attention_weights(s["dims"], s["q_abs"], s["lse"], s["latent_cache"], s["rope_cache"], s["page_table"],
                          s["seq_lens"], s["weights_in"], s["weights"], s["workspace"])
    return s["weights"]


def _own_evict(s):
    from mlra_latent_kv_b200 import abi
    abi.latent_evict(s["dims"], s["case"]["recent"], s["evict_pages"], s["weights_in"], s["page_table"],
                     s["seq_lens"], s["latent_cache"], s["rope_cache"], s["weights"], s["page_table_out"],
                     s["seq_lens_out"], s["workspace"])
    return {k: s[k] for k in ("latent_cache", "rope_cache", "weights", "page_table_out", "seq_lens_out")}


def _rotate(x, pos, dtype):
    """RoPE of x [..., d_r] at positions pos (broadcast over the rest): interleaved pairs, angles in 64 bits."""
    d_r = x.shape[-1]
    theta = ROPE_BASE ** (-torch.arange(0, d_r, 2, device=x.device, dtype=torch.float64) / d_r)
    angle = pos.double()[..., None] * theta
    c, s = torch.cos(angle).to(dtype), torch.sin(angle).to(dtype)
    x0, x1 = x[..., 0::2].to(dtype), x[..., 1::2].to(dtype)
    return torch.stack((x0 * c - x1 * s, x0 * s + x1 * c), -1).flatten(-2)


def _plain_prompt(s):
    """Scores of the padded batch as two products (content, rotary), softmax over the keys up to each query's own."""
    H, d_v = s["out"].shape[1:]
    kv = s["k_nope"].shape[1]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    B, (Lq, Lk) = cu_q.numel() - 1, s["longest"]
    q_len, k_len = cu_q.diff()[:, None], cu_k.diff()[:, None]
    iq, ik = torch.arange(Lq, device="cuda")[None], torch.arange(Lk, device="cuda")[None]
    at_q = (cu_q[:-1, None] + iq).clamp_max(s["q_nope"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp_max(s["k_nope"].shape[0] - 1)
    pos = k_len - q_len + iq                                                     # a query's own position
    q = s["q_nope"].float()[at_q].view(B, Lq, kv, H // kv, -1).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = s["k_nope"].float()[at_k].permute(0, 2, 3, 1)                            # [B, kv, d_h, Lk]
    x = (q @ k).view(B, H, Lq, Lk)
    q_rot = _rotate(s["q_rope"][at_q], pos[:, :, None], torch.float32).transpose(1, 2)
    page = s["page_table"].clamp_min(0).long()[:, ik[0] // PAGE]
    k_rot = s["rope_cache"].float()[page, ik % PAGE]                             # [B, Lk, d_r]
    x += (q_rot.reshape(B, H * Lq, -1) @ k_rot.transpose(1, 2)).view(B, H, Lq, Lk)
    x *= s["scale"]
    x.masked_fill_(~((ik[:, None, :] <= pos[:, :, None]) & (ik < k_len)[:, None, :])[:, None], float("-inf"))
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    v = torch.where((ik < k_len)[:, :, None, None], s["v"].float()[at_k], 0.0).permute(0, 2, 1, 3)
    o = (p.view(B, kv, H // kv * Lq, Lk) @ v).view(B, H, Lq, d_v) / p.sum(-1, keepdim=True)
    return o.transpose(1, 2)[iq < q_len].to(s["out"].dtype)                      # the packed rows


def _plain_absorb(s):
    lat = torch.einsum("bhd,hdc->bhc", s["q_nope"].float(), s["W_UK"].float())
    rot = _rotate(s["q_rope"], s["q_pos"][:, None], torch.float32)
    return (torch.cat((lat, rot), -1) * (s["scale"] * LOG2E)).to(s["q_abs"].dtype)


def _scores(s):
    """Base-2 logits [B, branches, H, slots] of the absorbed query against the cache (NaN in slots nobody wrote)."""
    nb, (B, maxp) = s["case"]["branches"], s["page_table"].shape
    page = s["page_table"].clamp_min(0).long()
    lat = s["latent_cache"][page].float().view(B, maxp * PAGE, nb, -1)
    q = s["q_abs"].float()
    q_lat = q[..., :-s["rope_cache"].shape[-1]].view(B, q.shape[1], nb, -1).permute(0, 2, 1, 3)
    x = q_lat @ lat.permute(0, 2, 3, 1)
    rope = s["rope_cache"][page].float().view(B, maxp * PAGE, -1)
    return x.add_((q[..., -rope.shape[-1]:] @ rope.transpose(1, 2))[:, None])


def _plain_weights(s):
    p = _scores(s).sub_(s["lse"][..., None]).exp2_().sum((1, 2))
    valid = torch.arange(p.shape[1], device="cuda")[None, :] < s["seq_lens"][:, None]
    return torch.where(valid, s["weights_in"] + p, s["weights"])


def _plain_evict(s):
    w, table, L = s["weights_in"], s["page_table"].long(), s["seq_lens"].long()[:, None]
    n = s["evict_pages"].long()[:, None]
    slots = w.shape[1]
    slot = torch.arange(slots, device="cuda")[None, :].expand_as(w)
    # those that may go, least weight first, of equal ones the later slot first
    rev = slot.flip(1)
    order = rev.gather(1, torch.argsort(w.nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
                                        .gather(1, rev), dim=1, stable=True))
    barred = order >= L - s["case"]["recent"]
    order = order.gather(1, torch.argsort(barred.to(torch.uint8), dim=1, stable=True))
    gone = torch.zeros_like(w, dtype=torch.bool).scatter_(1, order, slot < n * PAGE)
    # what stays of the first n pages moves into the slots that become free behind them
    src = torch.nonzero((slot < n * PAGE) & ~gone).unbind(1)
    dst = torch.nonzero((slot >= n * PAGE) & gone).unbind(1)
    for pool in (s["latent_cache"], s["rope_cache"]):
        pool[table[dst[0], dst[1] // PAGE], dst[1] % PAGE] = pool[table[src[0], src[1] // PAGE], src[1] % PAGE]
    w = w.clone()
    w[dst] = w[src]
    moved = slot + n * PAGE
    weights = torch.where(moved < L, w.gather(1, moved.clamp_max(slots - 1)), 0.0)
    page = torch.arange(table.shape[1], device="cuda")[None, :] + n
    table_out = torch.where(page < table.shape[1], table.gather(1, page.clamp_max(table.shape[1] - 1)), -1)
    return {"latent_cache": s["latent_cache"], "rope_cache": s["rope_cache"], "weights": weights,
            "page_table_out": table_out.int(), "seq_lens_out": (L - n * PAGE)[:, 0].int()}


_RUN_PLAIN = {"prompt": _plain_prompt, "absorb": _plain_absorb, "weights": _plain_weights, "evict": _plain_evict}
_RUN_OWN = {"prompt": _own_prompt, "absorb": _own_absorb, "weights": _own_weights, "evict": _own_evict}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits, one sequence (and head) at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "absorb": _exact_absorb, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](s)


def _turn(x, pos):
    """Each pair (x0, x1) of the last axis as a complex number, turned by pos * base^(-2i/d_r)."""
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], -1, 2).contiguous())
    i = torch.arange(z.shape[-1], device=x.device, dtype=torch.float64)
    angle = pos.double()[..., None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device=x.device),
                                                -2 * i / x.shape[-1])
    return torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)).flatten(-2)


def _tokens(pool, row, n):
    return pool[row[:-(-n // PAGE)].long()].flatten(0, 1)[:n].double() if n else pool[:0].flatten(0, 1).double()


def _exact_prompt(s):
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    T, H, d_v = s["out"].shape
    group = H // s["k_nope"].shape[1]
    out = torch.zeros(T, H, d_v, dtype=torch.float64, device="cuda")
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        at = torch.arange(m - n, m, device="cuda")
        rope = _tokens(s["rope_cache"], s["page_table"][b], m)
        past = torch.arange(m, device="cuda")[None, :] > at[:, None]
        for h in range(H):
            rows = slice(cu_q[b], cu_q[b + 1])
            query = torch.cat((s["q_nope"][rows, h].double(), _turn(s["q_rope"][rows, h], at)), 1)
            key = torch.cat((s["k_nope"][cu_k[b]:cu_k[b + 1], h // group].double(), rope), 1)
            logit = (s["scale"] * query @ key.T).masked_fill(past, -math.inf)
            out[rows, h] = torch.softmax(logit, 1) @ s["v"][cu_k[b]:cu_k[b + 1], h // group].double()
    return out


def _exact_absorb(s):
    q = s["q_nope"].double().transpose(0, 1) @ s["W_UK"].double()                # [H, B, d_c]
    turned = _turn(s["q_rope"].transpose(0, 1), s["q_pos"][None, :])
    return (s["scale"] / math.log(2) * torch.cat((q, turned), 2)).transpose(0, 1).contiguous()


def _exact_weights(s):
    out = s["weights"].double()
    d_c = s["latent_cache"].shape[-1]
    nb = s["case"]["branches"]
    for b, n in enumerate(s["seq_lens"].tolist()):
        c, k = _tokens(s["latent_cache"], s["page_table"][b], n), _tokens(s["rope_cache"], s["page_table"][b], n)
        q = s["q_abs"][b].double()
        total = s["weights_in"][b, :n].double()
        for r in range(nb):
            cols = slice(r * d_c // nb, (r + 1) * d_c // nb)
            logit = torch.cat((c[:, cols], k), 1) @ torch.cat((q[:, cols], q[:, d_c:]), 1).T
            total = total + torch.pow(2.0, logit - s["lse"][b, r].double()).sum(1)
        out[b, :n] = total
    return out


def _exact_evict(s):
    """Whole numbers and copies: by sorting each sequence's tokens on the host."""
    lat, rope = s["latent_cache"], s["rope_cache"]
    weights, table_out, lens_out = [], [], []
    slots = s["weights_in"].shape[1]
    for b, (n, p) in enumerate(zip(s["seq_lens"].tolist(), s["evict_pages"].tolist())):
        row, w = s["page_table"][b].tolist(), s["weights_in"][b].tolist()
        free = p * PAGE
        gone = set(sorted(range(max(0, n - s["case"]["recent"])), key=lambda t: (w[t], -t))[:free])
        src = [t for t in range(free) if t not in gone]
        dst = [t for t in range(free, n) if t in gone]
        page = s["page_table"][b].long()
        i, j = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (src, dst))
        for pool in (lat, rope):
            pool[page[j // PAGE], j % PAGE] = pool[page[i // PAGE], i % PAGE].clone()
        for t, u in zip(src, dst):
            w[u] = w[t]
        weights.append(w[free:n] + [0.0] * (slots - (n - free)))
        table_out.append(row[p:] + [-1] * p)
        lens_out.append(n - free)
    return {"latent_cache": lat, "rope_cache": rope, "weights": torch.tensor(weights, dtype=torch.float64),
            "page_table_out": _int(table_out), "seq_lens_out": _int(lens_out)}
