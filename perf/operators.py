"""The operators of a bounded, paged key-value cache, as cases to measure.

``paged_decode``   attention of one new token over the cache, with or without
                   the running sum of each cached token's attention weight;
``cache_append``   new tokens' keys and values into the cache's pages;
``cache_evict``    the cache cut to a budget of tokens by accumulated weight;
``key_weights``    the accumulated attention weight of a prompt's keys.

Layouts: a cache is [pages, kv heads, page size, d] of 16-bit floats; slot j of
sequence b lies in page table[b, j // page size]; weights (float32) and
positions (int32) are [B, kv heads, L] with L = table width * page size.
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _decode(name, B, Hq, Hkv, n, d, ps, dtype="bf16", weights=False, ragged=False, q_std=1.0):
    return {"name": name, "op": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "n": n, "d": d, "ps": ps,
            "dtype": dtype, "weights": weights, "ragged": ragged, "q_std": q_std}


def _append(name, B, Hkv, n, new, d, ps, dtype="bf16", ragged=False):
    return {"name": name, "op": "append", "B": B, "Hkv": Hkv, "n": n, "new": new, "d": d, "ps": ps,
            "dtype": dtype, "ragged": ragged}


def _evict(name, B, Hkv, n, budget, recent, d, ps, dtype="bf16", ragged=False):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "n": n, "budget": budget,
            "recent": recent, "d": d, "ps": ps, "dtype": dtype, "ragged": ragged}


def _keyw(name, B, Hq, Hkv, N, d, causal=True, dtype="bf16", padded=False, q_std=1.0):
    return {"name": name, "op": "key_weights", "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d,
            "causal": causal, "dtype": dtype, "padded": padded, "q_std": q_std}


def listed():
    return [
        # one user's chat, a short context: latency is all that counts
        _decode("decode_b1_h32kv8_n512_d128", 1, 32, 8, 512, 128, 16),
        # one long document, few heads (B=1 H=2 N=16384): only a split over the length fills the GPU
        _decode("decode_b1_h2_n16384_d128_w", 1, 2, 2, 16384, 128, 64, weights=True),
        # a served batch of uneven contexts, shared key heads, weights kept for a later eviction
        _decode("decode_b32_h32kv8_n8192_d128_w", 32, 32, 8, 8192, 128, 16, weights=True,
                ragged=True, q_std=3.0),
        # the half-size heads in the other 16-bit type, every query head with keys of its own
        _decode("decode_b16_h16_n2047_d64_fp16", 16, 16, 16, 2047, 64, 32, dtype="fp16"),
        # every step of a served batch writes one token a sequence
        _append("append_b32_kv8_new1_d128", 32, 8, 2047, 1, 128, 16, ragged=True),
        # prompts of uneven length in one padded batch go into the cache
        _append("append_b4_kv32_new8192_d128", 4, 32, 0, 8192, 128, 16, ragged=True),
        # steady state of a bounded cache: one token over the budget
        _evict("evict_b32_kv8_n2049_to2048_d128", 32, 8, 2049, 2048, 256, 128, 16),
        # a prompt is cut to a quarter
        _evict("evict_b4_kv32_n8192_to2048_d128", 4, 32, 8192, 2048, 512, 128, 16),
        # one long prompt, few heads: the selection itself is the work
        _evict("evict_b1_kv2_n16384_to4095_d64", 1, 2, 16384, 4095, 100, 64, 64, dtype="fp16"),
        # weights of a small prompt batch
        _keyw("key_weights_b2h4_n1024_d64", 2, 4, 4, 1024, 64),
        # the middle workload, uneven prompts in a padded batch, key heads shared by four
        _keyw("key_weights_b8h16kv4_n2048_d128", 8, 16, 4, 2048, 128, padded=True),
        # long prompts with sharp softmax rows
        _keyw("key_weights_b2h16_n8192_d128", 2, 16, 16, 8192, 128, q_std=3.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "evict", "evict", "key_weights", "key_weights"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    ps = rng.choice([8, 16, 24, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    B = _log_int(rng, 1, 48)
    ragged = rng.random() < 0.6
    if op == "decode":
        n = _log_int(rng, 1, 16384)
        while B * Hkv * n * d > 32 * 8 * 4700 * 128 or B * Hkv * group * n > 32 * 32 * 4700:
            B, n = max(1, B // 2), max(1, n - n // 3)
        c = _decode("", B, Hkv * group, Hkv, n, d, ps, dtype, rng.random() < 0.5, ragged,
                    rng.choice([1.0, 2.0, 3.0]))
    elif op == "append":
        n, new = rng.choice([0, _log_int(rng, 1, 4096)]), rng.choice([1, _log_int(rng, 1, 8192)])
        while B * Hkv * (n + new) * d > 4 * 32 * 8192 * 128 // 2:
            B, new, n = max(1, B // 2), max(1, new - new // 3), n // 2
        c = _append("", B, Hkv, n, new, d, ps, dtype, ragged)
    elif op == "evict":
        n = _log_int(rng, 2, 20000)
        while B * Hkv * n * d > 4 * 32 * 8192 * 128 // 2:
            B, n = max(1, B // 2), max(2, n - n // 3)
        budget = rng.randint(1, n)
        c = _evict("", B, Hkv, n, budget, rng.randint(0, budget), d, ps, dtype, ragged)
    else:
        N = _log_int(rng, 16, 8192)
        causal = rng.random() < 0.7
        B = min(B, 8)
        while B * Hkv * group * N * N * d > 2 * 16 * 8192 * 8192 * 128 // 2:
            B, N = max(1, B // 2), max(1, N - N // 4)
        c = _keyw("", B, Hkv * group, Hkv, N, d, causal, dtype, causal and ragged,
                  rng.choice([1.0, 3.0]))
    del c["name"]
    return c


def _lengths(case, most, least):
    """The sequences' lengths: all `most`, or uneven ones that the case's sizes fix."""
    B = case["B"]
    uneven = case.get("ragged") or case.get("padded")
    if not uneven:
        return [most] * B
    r = random.Random(B * 1000003 + most)
    return [max(least, min(most, int(most * r.uniform(0.15, 1.0)))) for _ in range(B - 1)] + [most]


def _case_lens(case):
    """(tokens in the cache, new tokens) of each sequence."""
    B = case["B"]
    if case["op"] == "append":
        return [case["n"]] * B, _lengths(case, case["new"], 1)
    return _lengths(case, case["n"], 1), [0] * B


def _moves(n, k, recent):
    """Rows that an eviction moves on average, weights being in no order."""
    if n <= k:
        return 0.0
    if n == recent:
        return 0.0
    stay = (k - recent) * min(1.0, k / (n - recent)) if k <= n - recent else \
        (k - recent) + (k - (n - recent))
    return k - stay


def work(case):
    B, d, op = case["B"], case["d"], case["op"]
    if op == "key_weights":
        Hq, Hkv, N = case["Hq"], case["Hkv"], case["N"]
        qn = _lengths(case, N, 1)
        pairs = sum(m * (m + 1) / 2 if case["causal"] else m * N for m in qn)
        return {"bytes": sum(qn) * Hq * (2 * d + 4) + B * Hkv * N * (2 * d + 4),
                "flops": 2.0 * Hq * d * pairs}
    Hkv = case["Hkv"]
    lens, new = _case_lens(case)
    if op == "decode":
        tok = sum(lens) * Hkv
        return {"bytes": tok * 4 * d + B * case["Hq"] * (4 * d + 4) + (8 * tok if case["weights"] else 0),
                "flops": 4.0 * sum(lens) * case["Hq"] * d}
    if op == "append":
        tok = sum(new) * Hkv
        return {"bytes": tok * (8 * d + 4 + 8), "flops": 0}
    moved = sum(_moves(n, case["budget"], case["recent"]) for n in lens) * Hkv
    kept = sum(min(n, case["budget"]) for n in lens) * Hkv
    return {"bytes": sum(lens) * Hkv * 8 + moved * 8 * d + kept * 8, "flops": 0}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, d, dt = case["B"], case["d"], DT[case["dtype"]]

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case}
    if case["op"] == "key_weights":
        Hq, Hkv, N = case["Hq"], case["Hkv"], case["N"]
        s["q"], s["k"] = randn(B, Hq, N, d, std=case["q_std"]), randn(B, Hkv, N, d)
        s["q_lens"] = ints(_lengths(case, N, 1)) if case["padded"] else None
        s["out"] = torch.empty(B, Hkv, N, device="cuda")
        # the forward pass's logsumexp, head by head
        s["lse"] = torch.empty(B, Hq, N, device="cuda")
        for b in range(B):
            for h in range(Hq):
                t = (s["q"][b, h].float() @ s["k"][b, h * Hkv // Hq].float().T).mul_(d ** -0.5)
                if case["causal"]:
                    t += torch.full((N, N), -math.inf, device="cuda").triu_(1)
                s["lse"][b, h] = torch.logsumexp(t, -1)
        return s
    Hkv, ps = case["Hkv"], case["ps"]
    lens, new = _case_lens(case)
    width = max(1, -(-max(a + b for a, b in zip(lens, new)) // ps))
    pages = B * width + 3
    L = width * ps
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * width].to(torch.int32).view(B, width)
    s["k_cache"], s["v_cache"] = randn(pages, Hkv, ps, d), randn(pages, Hkv, ps, d)
    s["lens"] = ints(lens)
    if case["op"] == "decode":
        s["q"] = randn(B, case["Hq"], d, std=case["q_std"])
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, case["Hq"], device="cuda")
        if case["weights"]:  # sums over earlier tokens: a long tail
            s["weights"] = torch.empty(B, Hkv, L, device="cuda").log_normal_(0.0, 1.5, generator=g)
            s["weights_out"] = torch.zeros(B, Hkv, L, device="cuda")
    elif case["op"] == "append":
        T = max(new)
        s["k"], s["v"] = randn(B, Hkv, T, d), randn(B, Hkv, T, d)
        s["new_weights"] = torch.empty(B, Hkv, T, device="cuda").log_normal_(0.0, 1.5, generator=g)
        s["num_new"] = ints(new)
        s["next_pos"] = s["lens"] + 5  # some tokens were evicted before
        s["weights"] = torch.zeros(B, Hkv, L, device="cuda")
        s["positions"] = torch.zeros(B, Hkv, L, dtype=torch.int32, device="cuda")
        s["lens_out"] = torch.empty_like(s["lens"])
    else:
        w = torch.empty(B, Hkv, L, device="cuda").log_normal_(0.0, 1.5, generator=g)
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.05] = 0.0  # tokens that nothing looked at
        s["weights"] = w
        s["positions"] = torch.arange(L, dtype=torch.int32, device="cuda").expand(B, Hkv, L).contiguous()
        s["next_pos"] = s["lens"].clone()
        s["weights_out"] = torch.zeros_like(w)
        s["positions_out"] = torch.zeros_like(s["positions"])
        s["lens_out"] = torch.empty_like(s["lens"])
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    if op == "decode":
        return _plain_decode(s)
    if op == "append":
        return _plain_append(s)
    if op == "evict":
        return _plain_evict(s)
    return _plain_key_weights(s)


def _own(op, s):
    import exact_attention_64_gb300 as fa2

    if op == "decode":
        w, w_out = s.get("weights"), s.get("weights_out")
        o, lse = fa2.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                  weights=w, weights_out=w_out, out=s["o"], lse=s["lse"])
        return {"o": o, "lse": lse} if w is None else {"o": o, "lse": lse, "weights": w_out}
    if op == "append":
        lens = fa2.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                num_new=s["num_new"], weights=s["weights"],
                                new_weights=s["new_weights"], positions=s["positions"],
                                next_pos=s["next_pos"], lens_out=s["lens_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"],
                "positions": s["positions"], "lens": lens}
    if op == "evict":
        c = s["case"]
        lens = fa2.cache_evict(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["weights"],
                               c["budget"], recent=c["recent"], positions=s["positions"],
                               next_pos=s["next_pos"], weights_out=s["weights_out"],
                               positions_out=s["positions_out"], lens_out=s["lens_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights_out"],
                "positions": s["positions_out"], "lens": lens}
    return fa2.key_weights(s["q"], s["k"], s["lse"], causal=s["case"]["causal"],
                           q_lens=s["q_lens"], out=s["out"])


def _rows(s, slots):
    """Rows of the flattened cache that slots [B, Hkv, M] lie in."""
    Hkv, ps = s["case"]["Hkv"], s["case"]["ps"]
    page = torch.gather(s["table"].long().unsqueeze(1).expand(-1, Hkv, -1), 2, slots // ps)
    head = torch.arange(Hkv, device="cuda").view(1, Hkv, 1)
    return (page * Hkv + head) * ps + slots % ps


def _all_slots(s):
    B, Hkv, L = s["case"]["B"], s["case"]["Hkv"], s["table"].shape[1] * s["case"]["ps"]
    return torch.arange(L, device="cuda").expand(B, Hkv, L)


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    slots = _all_slots(s)
    rows = _rows(s, slots)
    inside = (slots < s["lens"].view(B, 1, 1)).unsqueeze(2)  # [B, Hkv, 1, L]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    k = s["k_cache"].view(-1, d)[rows].float()
    t = (q @ k.transpose(-1, -2)) * d ** -0.5
    del k
    t = torch.where(inside, t, torch.full_like(t, -math.inf))
    m = t.amax(-1, keepdim=True)
    e = torch.exp(t - m)
    l = e.sum(-1, keepdim=True)
    p = e / l
    o = p @ s["v_cache"].view(-1, d)[rows].float()
    lse = (m + torch.log(l)).view(B, Hq)
    o = o.view(B, Hq, d).to(s["q"].dtype)
    if not c["weights"]:
        return {"o": o, "lse": lse}
    w = torch.where(inside.squeeze(2), s["weights"] + p.sum(2), s["weights_out"])
    return {"o": o, "lse": lse, "weights": w}


def _plain_append(s):
    c = s["case"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    T = s["k"].shape[2]
    i = torch.arange(T, device="cuda").expand(B, Hkv, T)
    fresh = i < s["num_new"].view(B, 1, 1)
    slots = torch.where(fresh, s["lens"].view(B, 1, 1) + i, torch.zeros_like(i))
    rows = _rows(s, slots)[fresh]
    s["k_cache"].view(-1, d)[rows] = s["k"][fresh]
    s["v_cache"].view(-1, d)[rows] = s["v"][fresh]
    b = torch.arange(B, device="cuda").view(B, 1, 1).expand_as(i)[fresh]
    h = torch.arange(Hkv, device="cuda").view(1, Hkv, 1).expand_as(i)[fresh]
    s["weights"][b, h, slots[fresh]] = s["new_weights"][fresh]
    s["positions"][b, h, slots[fresh]] = (s["next_pos"].view(B, 1, 1) + i).int()[fresh]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"],
            "positions": s["positions"], "lens": s["lens"] + s["num_new"]}


def _plain_evict(s):
    c = s["case"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    slots = _all_slots(s)
    L = slots.shape[-1]
    n = s["lens"].long().view(B, 1, 1)
    left = n.clamp(max=c["budget"])
    key = torch.where(s["positions"] >= (s["next_pos"] - c["recent"]).view(B, 1, 1),
                      torch.full_like(s["weights"], math.inf), s["weights"])
    key = torch.where(slots < n, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # ties: lowest slot first
    keep = torch.zeros_like(slots, dtype=torch.bool).scatter(2, order, slots < left)
    hole, mover = ~keep & (slots < left), keep & (slots >= left)
    # mover of each rank, then the source of every slot that is left
    rank = torch.where(mover, mover.cumsum(-1) - 1, torch.full_like(slots, L))
    of_rank = torch.zeros(B, Hkv, L + 1, dtype=torch.long, device="cuda").scatter(2, rank, slots)
    source = torch.where(hole, torch.gather(of_rank, 2, hole.cumsum(-1).sub(1).clamp(min=0)), slots)
    rows, dst = _rows(s, source), _rows(s, slots)
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.view(-1, d)
        flat[dst] = flat[rows]
    w = torch.where(slots < left, torch.gather(s["weights"], 2, source), s["weights_out"])
    p = torch.where(slots < left, torch.gather(s["positions"], 2, source), s["positions_out"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": w, "positions": p,
            "lens": s["lens"].clamp(max=c["budget"])}


def _plain_key_weights(s):
    c = s["case"]
    B, Hq, Hkv, N, d = c["B"], c["Hq"], c["Hkv"], c["N"], c["d"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, N, d)
    lse = s["lse"].view(B, Hkv, Hq // Hkv, N, 1)
    if s["q_lens"] is not None:  # padded queries have no weight
        off = (torch.arange(N, device="cuda") >= s["q_lens"].view(B, 1, 1, 1)).unsqueeze(-1)
        lse = torch.where(off, torch.full_like(lse, math.inf), lse)
    t = q @ (s["k"].float() * d ** -0.5).transpose(-1, -2).unsqueeze(2)
    t.sub_(lse).exp_()
    if c["causal"]:
        t.tril_()
    return t.sum(-2).sum(2)


# --------------------------------------------------------------------------
# The definition in 64 bits, one sequence at a time
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "key_weights":
        return _exact_key_weights(case, s)
    B, Hkv, ps, d = case["B"], case["Hkv"], case["ps"], case["d"]
    lens, new = _case_lens(case)

    def tokens(cache, b, n):  # [Hkv, n, d]
        return cache[s["table"][b].long()].transpose(0, 1).reshape(Hkv, -1, d)[:, :n]

    if op == "decode":
        Hq = case["Hq"]
        o = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        w = s["weights_out"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            k, v = tokens(s["k_cache"], b, n).double(), tokens(s["v_cache"], b, n).double()
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                t = (k[kv] * s["q"][b, h].double()).sum(-1) / math.sqrt(d)
                lse[b, h] = torch.logsumexp(t, 0)
                p = torch.exp(t - lse[b, h])
                o[b, h] = (p.unsqueeze(-1) * v[kv]).sum(0)
                if w is not None:
                    if h % (Hq // Hkv) == 0:
                        w[b, kv, :n] = s["weights"][b, kv, :n].double()
                    w[b, kv, :n] += p
        return {"o": o, "lse": lse} if w is None else {"o": o, "lse": lse, "weights": w}
    # Copies: worked out slot by slot on the host, one sequence and head at a time.
    table = s["table"].cpu().numpy().astype(np.int64)
    weights = s["weights" if op == "append" else "weights_out"].cpu().numpy().copy()
    positions = s["positions" if op == "append" else "positions_out"].cpu().numpy().copy()
    src_rows, dst_rows = [], []
    if op == "append":
        nw, start = s["new_weights"].cpu().numpy(), s["next_pos"].cpu().numpy()
        T = nw.shape[2]
        for b in range(B):
            at = np.arange(lens[b], lens[b] + new[b])
            for h in range(Hkv):
                dst_rows.append((table[b, at // ps] * Hkv + h) * ps + at % ps)
                src_rows.append((b * Hkv + h) * T + np.arange(new[b]))
                weights[b, h, at] = nw[b, h, :new[b]]
                positions[b, h, at] = start[b] + np.arange(new[b])
        left = [a + b for a, b in zip(lens, new)]
    else:
        w_in, p_in = s["weights"].cpu().numpy(), s["positions"].cpu().numpy()
        first = s["next_pos"].cpu().numpy() - case["recent"]
        left = [min(n, case["budget"]) for n in lens]
        for b in range(B):
            n, k = lens[b], left[b]
            for h in range(Hkv):
                w, p = w_in[b, h, :n], p_in[b, h, :n]
                order = np.lexsort((np.arange(n), -w.astype(np.float64), p < first[b]))
                kept = np.sort(order[:k])
                place = np.arange(k)
                free = np.setdiff1d(place, kept, assume_unique=True)
                place[free] = kept[kept >= k]
                weights[b, h, :k], positions[b, h, :k] = w[place], p[place]
                src_rows.append((table[b, place[free] // ps] * Hkv + h) * ps + place[free] % ps)
                dst_rows.append((table[b, free // ps] * Hkv + h) * ps + free % ps)
    src = torch.from_numpy(np.concatenate(src_rows)).cuda()
    dst = torch.from_numpy(np.concatenate(dst_rows)).cuda()
    caches = []
    for new_rows, cache in ((s.get("k"), s["k_cache"]), (s.get("v"), s["v_cache"])):
        flat = cache.view(-1, d)
        flat.index_copy_(0, dst, (flat if new_rows is None else new_rows.view(-1, d)).index_select(0, src))
        caches.append(cache)
    return {"k_cache": caches[0], "v_cache": caches[1], "weights": torch.from_numpy(weights),
            "positions": torch.from_numpy(positions),
            "lens": torch.tensor(left, dtype=torch.int32)}


def _exact_key_weights(case, s):
    B, Hq, Hkv, N, d = case["B"], case["Hq"], case["Hkv"], case["N"], case["d"]
    qn = _lengths(case, N, 1)
    out = torch.zeros(B, Hkv, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            k = s["k"][b, kv].double() / math.sqrt(d)
            for i in range(0, qn[b], 2048):
                j = min(qn[b], i + 2048)
                p = torch.exp(s["q"][b, h, i:j].double() @ k.T - s["lse"][b, h, i:j, None].double())
                if case["causal"]:
                    p = torch.where(torch.arange(N, device="cuda") <= torch.arange(i, j, device="cuda")[:, None],
                                    p, torch.zeros_like(p))
                out[b, kv] += p.sum(0)
    return out
