"""Operators around attention and its paged key-value cache, as cases to measure.

``rotary``         queries and keys of a projection turned by their positions,
                   optionally normed per head in the same pass, into the layout
                   that attention takes; and its backward pass;
``prefix_decode``  attention of one new token per sequence over a paged cache
                   whose sequences all begin with the same slots;
``cache_resize``   the page tables brought from one set of lengths to another.

Layouts: projections are [B, N, heads, d] (q, k and v side by side), attention's
tensors [B, heads, N, d]; a cache is [pages, kv heads, page size, d] of 16-bit
floats, and slot j of sequence b lies in page table[b, j // page size].
"""

import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _rotary(name, B, Hq, Hkv, N, d, r, dtype="bf16", interleaved=False, norm=None, start=0, scaled=False,
            backward=False):
    """r: turned elements of a head; norm: type of the norm's weights or None; start: the first position."""
    return {"name": name, "op": "rotary_bwd" if backward else "rotary", "B": B, "Hq": Hq, "Hkv": Hkv, "N": N,
            "d": d, "r": r, "dtype": dtype, "interleaved": interleaved, "norm": norm or "", "start": start,
            "scaled": scaled}


def _prefix(name, B, Hq, Hkv, shared, n, d, ps, dtype="bf16", q_std=1.0, strangers=0):
    """shared: slots that all begin with; n: most slots of a sequence behind them; strangers: sequences
    that are shorter than the prefix and have nothing of it."""
    return {"name": name, "op": "prefix", "B": B, "Hq": Hq, "Hkv": Hkv, "shared": shared, "n": n, "d": d,
            "ps": ps, "dtype": dtype, "q_std": q_std, "strangers": strangers}


def _resize(name, B, n, ps, churn, shared=0):
    """churn: share of the sequences that end, begin or are cut; the others grow by one slot.
    shared: first pages that all sequences name."""
    return {"name": name, "op": "resize", "B": B, "n": n, "ps": ps, "churn": churn, "shared": shared}


def listed():
    return [
        # one user's chat: the new token's queries and keys before they go to the cache; latency is all that counts
        _rotary("rotary_b1_h32kv8_n1_d128_norm", 1, 32, 8, 1, 128, 128, norm="fp32", start=30000, scaled=True),
        # one step of a served batch, every sequence at a position of its own
        _rotary("rotary_b32_h32kv8_n1_d128", 32, 32, 8, 1, 128, 128, start=8000, scaled=True),
        # prompts of the middle workload, key heads shared by four, normed, a quarter of the head turned
        _rotary("rotary_b8_h16kv4_n2047_d64_r16_norm_fp16", 8, 16, 4, 2047, 64, 16, dtype="fp16", interleaved=True,
                norm="fp16"),
        # the largest training workload, normed
        _rotary("rotary_b4_h32_n8192_d128_norm", 4, 32, 32, 8192, 128, 128, norm="bf16"),
        # its gradients, without and with the norm
        _rotary("rotary_bwd_b4_h32_n8192_d128", 4, 32, 32, 8192, 128, 128, backward=True),
        _rotary("rotary_bwd_b8_h16kv4_n2048_d128_norm", 8, 16, 4, 2048, 128, 64, norm="fp32", backward=True),
        # a few chats behind one system prompt
        _prefix("prefix_decode_b8_h32kv8_p2000_n300_d128", 8, 32, 8, 2000, 300, 128, 16),
        # two heads' long document, a few questions about it
        _prefix("prefix_decode_b5_h2_p16384_n63_d64_fp16", 5, 2, 2, 16384, 63, 64, 64, dtype="fp16"),
        # a served batch behind a long prompt, contexts of uneven length
        _prefix("prefix_decode_b64_h32kv8_p8192_n1024_d128", 64, 32, 8, 8192, 1024, 128, 16, q_std=2.0, strangers=2),
        # many samples of one long prompt: the products count
        _prefix("prefix_decode_b256_h32kv8_p16384_n200_d128", 256, 32, 8, 16384, 200, 128, 64),
        # every step of a served batch: a new page for one sequence in sixteen
        _resize("cache_resize_b256_n8192_step", 256, 8192, 16, 0.0),
        # requests come, end and are cut back to a budget
        _resize("cache_resize_b512_n16384_churn", 512, 16384, 16, 0.75, shared=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_bwd", "prefix", "prefix", "resize"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 8])
    if op in ("rotary", "rotary_bwd"):
        B, N = _log_int(rng, 1, 64), rng.choice([1, _log_int(rng, 2, 16384)])
        if op == "rotary_bwd":
            N = _log_int(rng, 16, 16384)
        while B * N * Hkv * (group + 1) * d > 4 * 64 * 8192 * 128 // 2:
            B, N = max(1, B // 2), max(1, N - N // 3)
        c = _rotary("", B, Hkv * group, Hkv, N, d, 16 * rng.randint(1, d // 16), dtype, rng.random() < 0.5,
                    rng.choice([None, dtype, "fp32"]), rng.choice([0, _log_int(rng, 1, 2000000)]),
                    rng.random() < 0.5, op == "rotary_bwd")
    elif op == "prefix":
        B, shared, n = _log_int(rng, 1, 256), _log_int(rng, 1, 32768), rng.choice([1, _log_int(rng, 1, 4096)])
        while B * Hkv * group * shared * d > 256 * 32 * 16384 * 128 // 2 or B * Hkv * group * n * d > 256 * 32 * 200 * 128:
            B, shared, n = max(1, B // 2), max(1, shared - shared // 3), max(1, n - n // 3)
        c = _prefix("", B, Hkv * group, Hkv, shared, n, d, rng.choice([1, 8, 16, 24, 32, 64, 128]), dtype,
                    rng.choice([1.0, 2.0, 3.0]), min(B - 1, rng.choice([0, 0, 1, 3])))
    else:
        B, n, ps = _log_int(rng, 1, 512), _log_int(rng, 1, 16384), rng.choice([1, 8, 16, 24, 64, 128])
        while B * n > 512 * 16384 // 16 * ps:
            B, n = max(1, B // 2), max(1, n - n // 3)
        c = _resize("", B, n, ps, rng.choice([0.0, 0.3, 0.9]), rng.randint(0, max(0, n // ps // 2)))
    del c["name"]
    return c


def _own_lens(case):
    """A prefix case: slots of each sequence (the shared ones among them)."""
    r = random.Random(case["B"] * 1000003 + case["n"])
    out = [case["shared"] + max(1, int(case["n"] * r.uniform(0.15, 1.0))) for _ in range(case["B"])]
    out[-1] = case["shared"] + case["n"]
    for i in range(case["strangers"]):
        out[i] = r.randint(0, min(case["shared"] - 1, case["n"]))
    return out


def _resize_lens(case):
    """A resize case: lengths before and after."""
    r = random.Random(case["B"] * 7919 + case["n"])
    old, new = [], []
    least = case["shared"] * case["ps"]  # pages that all name are neither taken nor given back
    for _ in range(case["B"]):
        n = r.randint(least, case["n"])
        u = r.random() / case["churn"] if case["churn"] > 0 else 2.0
        if u < 0.33:            # ends
            a, b = n, least
        elif u < 0.66:          # begins
            a, b = least, n
        elif u < 1.0:           # cut to a budget
            a, b = n, min(n, max(least, case["n"] // 4))
        else:                   # one more token
            a, b = n, min(n + 1, case["n"])
        old.append(a)
        new.append(b)
    return old, new


def work(case):
    op = case["op"]
    if op in ("rotary", "rotary_bwd"):
        el = case["B"] * case["N"] * (case["Hq"] + case["Hkv"]) * case["d"]
        norm = case["norm"] != ""
        per = 4 + (2 if norm and op == "rotary_bwd" else 0)
        return {"bytes": el * per + 4 * case["B"] + 4 * case["r"], "flops": el * (3 + 4 * norm)}
    if op == "prefix":
        d, Hq, Hkv, B = case["d"], case["Hq"], case["Hkv"], case["B"]
        lens = _own_lens(case)
        ends = [n - case["shared"] if n >= case["shared"] else n for n in lens]
        return {"bytes": (case["shared"] + sum(ends)) * Hkv * 4 * d + B * Hq * (4 * d + 4),
                "flops": 4.0 * sum(lens) * Hq * d}
    old, new = _resize_lens(case)
    ps = case["ps"]
    pages = sum(abs(-(-a // ps) - -(-b // ps)) for a, b in zip(old, new))
    # there and back: lengths in and out, and of each page its table entry, its count and its place in the list
    return {"bytes": 2 * (12 * case["B"] + pages * (4 + 8 + 4)), "flops": 0}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _frequencies(r, scaled):
    """Radians per position of each pair; scaled: the slow ones stretched to eight times the context."""
    f = 10000.0 ** (-np.arange(0, r, 2, dtype=np.float64) / r)
    if scaled:
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 3.0, 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return f


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dt=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op in ("rotary", "rotary_bwd"):
        B, Hq, Hkv, N, d, dt = case["B"], case["Hq"], case["Hkv"], case["N"], case["d"], DT[case["dtype"]]
        x = randn(B, N, Hq + 2 * Hkv, d, std=1.5, dt=dt)  # the projection's output
        s["q"], s["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["freqs"] = torch.from_numpy(_frequencies(case["r"], case["scaled"])).cuda()
        s["amplitude"] = 1.25 if case["scaled"] else 1.0
        # the first position of each sequence: its tokens follow one another
        s["positions"] = (case["start"] + torch.randint(0, 1 + case["start"] // 2, (B,), generator=g, device="cuda")).int()
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (randn(d, std=0.1).add_(1.0).to(DT[case["norm"]]) for _ in range(2))
        if op == "rotary_bwd":
            s["dq"], s["dk"] = randn(B, Hq, N, d, dt=dt), randn(B, Hkv, N, d, dt=dt)
        return s
    if op == "prefix":
        B, Hq, Hkv, d, ps, dt = case["B"], case["Hq"], case["Hkv"], case["d"], case["ps"], DT[case["dtype"]]
        lens, P = _own_lens(case), case["shared"]
        width, whole = -(-max(lens) // ps), P // ps
        own_pages = width - whole  # the prefix's last, partly filled page is every sequence's own
        pages = whole + B * own_pages + case["strangers"] * whole + 2
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.empty(B, width, dtype=torch.int32, device="cuda")
        table[:, :whole] = order[:whole]
        table[:, whole:] = order[whole:whole + B * own_pages].view(B, own_pages)
        if case["strangers"]:
            m = case["strangers"] * whole
            table[:case["strangers"], :whole] = order[pages - 2 - m:pages - 2].view(-1, whole)
        s["k_cache"], s["v_cache"] = randn(pages, Hkv, ps, d, dt=dt), randn(pages, Hkv, ps, d, dt=dt)
        if P % ps:  # each sequence's copy of that page
            first, rest = table[-1, whole].long(), table[case["strangers"]:, whole].long()
            for c in (s["k_cache"], s["v_cache"]):
                c[rest, :, :P % ps] = c[first, :, :P % ps].clone()
        s["table"], s["lens"] = table, ints(lens)
        s["prefix"] = table[-1, :-(-P // ps)].clone()
        s["prefix_len"] = ints([P])
        s["q"] = randn(B, Hq, d, std=case["q_std"], dt=dt)
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, Hq, device="cuda")
        return s
    B, n, ps, shared = case["B"], case["n"], case["ps"], case["shared"]
    old, new = _resize_lens(case)
    width = max(1, -(-n // ps))
    held = [max(shared, -(-a // ps)) for a in old]
    pages = shared + sum(h - shared for h in held) + sum(max(0, -(-b // ps) - -(-a // ps)) for a, b in zip(old, new)) + 7
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    mine = (col >= shared) & (col < ints(held).view(B, 1))
    table[:, :shared] = order[:shared]
    table[mine] = order[shared:shared + int(mine.sum())]
    used = shared + int(mine.sum())
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:shared].long()] = B
    refs[order[shared:used].long()] = 1
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - used] = order[used:]
    s.update(table=table, refs=refs, free=free, num_free=ints([pages - used]), lens=ints(old), new_lens=ints(new),
             there=torch.empty(B, dtype=torch.int32, device="cuda"), back=torch.empty(B, dtype=torch.int32, device="cuda"))
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    if op == "rotary":
        q, k = _plain_rotary(s, s["q"], s["q_weight"]), _plain_rotary(s, s["k"], s["k_weight"])
        return {"q": q, "k": k}
    if op == "rotary_bwd":
        out = {}
        out["q"], out["q_weight"] = _plain_rotary_bwd(s, s["dq"], s["q"], s["q_weight"])
        out["k"], out["k_weight"] = _plain_rotary_bwd(s, s["dk"], s["k"], s["k_weight"])
        return {n: t for n, t in out.items() if t is not None}
    if op == "prefix":
        return _plain_prefix(s)
    _plain_resize(s, s["lens"], s["new_lens"], s["there"])
    _plain_resize(s, s["there"], s["lens"], s["back"])
    return {n: s[n] for n in ("table", "refs", "free", "num_free", "there", "back")}


def _own(op, s):
    import exact_attention_64_gb300 as fa2

    c = s["case"]
    if op in ("rotary", "rotary_bwd"):
        kw = dict(positions=s["positions"], interleaved=c["interleaved"], q_weight=s["q_weight"],
                  k_weight=s["k_weight"], eps=EPS, amplitude=s["amplitude"])
        if op == "rotary":
            q, k = fa2.rotary_forward(s["q"], s["k"], s["freqs"], **kw)
            return {"q": q, "k": k}
        if not c["norm"]:
            q, k, _, _ = fa2.rotary_backward(s["dq"], s["dk"], s["freqs"], **kw)
            return {"q": q, "k": k}
        q, k, wq, wk = fa2.rotary_backward(s["dq"], s["dk"], s["freqs"], q=s["q"], k=s["k"], **kw)
        return {"q": q, "q_weight": wq, "k": k, "k_weight": wk}
    if op == "prefix":
        o, lse = fa2.prefix_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["prefix"],
                                   s["prefix_len"], out=s["o"], lse=s["lse"])
        return {"o": o, "lse": lse}
    for a, b, out in ((s["lens"], s["new_lens"], s["there"]), (s["there"], s["lens"], s["back"])):
        fa2.cache_resize(s["table"], a, b, s["refs"], s["free"], s["num_free"], c["ps"], lens_out=out)
    return {n: s[n] for n in ("table", "refs", "free", "num_free", "there", "back")}


def _turns(s):
    """cos and sin [B, 1, N, r / 2] in fp32 of angles formed in 64 bits."""
    N = s["case"]["N"]
    pos = s["positions"].double().view(-1, 1) + torch.arange(N, device="cuda", dtype=torch.float64)
    a = (pos.unsqueeze(-1) * s["freqs"]).unsqueeze(1)
    return (torch.cos(a) * s["amplitude"]).float(), (torch.sin(a) * s["amplitude"]).float()


def _halves(c):
    """Where the first and the second elements of the pairs stand."""
    r = c["r"]
    return (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))


def _plain_rotary(s, x, weight):
    c = s["case"]
    dt = x.dtype
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    cos, sin = _turns(s)
    first, second = _halves(c)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    y[..., c["r"]:] = x[..., c["r"]:]
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y.to(dt)


def _plain_rotary_bwd(s, dy, x, weight):
    c = s["case"]
    dt = dy.dtype
    dy = dy.float()
    cos, sin = _turns(s)
    first, second = _halves(c)
    g = torch.empty_like(dy)
    g[..., c["r"]:] = dy[..., c["r"]:]
    g[..., first] = dy[..., first] * cos + dy[..., second] * sin
    g[..., second] = dy[..., second] * cos - dy[..., first] * sin
    if weight is None:
        return g.to(dt), None
    x = x.float()
    inv = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * inv
    dw = (g * xh).sum((0, 1, 2))
    g = g * weight.float()
    dx = (g - xh * (g * xh).mean(-1, keepdim=True)) * inv
    return dx.to(dt), dw.to(weight.dtype)


def _rows(table, slots, head, Hkv, ps):
    """Rows of the flattened cache."""
    return (torch.gather(table.long(), -1, slots // ps) * Hkv + head) * ps + slots % ps


def _plain_prefix(s):
    c = s["case"]
    B, Hq, Hkv, d, ps, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["ps"], c["shared"]
    kc, vc = s["k_cache"].view(-1, d), s["v_cache"].view(-1, d)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d) * d ** -0.5
    n = s["lens"].long().view(B, 1, 1)
    has = n >= P
    head = torch.arange(Hkv, device="cuda").view(Hkv, 1)
    slots = torch.arange(P, device="cuda").expand(Hkv, P)
    rows = _rows(s["prefix"].expand(Hkv, -1), slots, head, Hkv, ps)
    tp = q.transpose(0, 1).reshape(Hkv, -1, d) @ kc[rows].float().transpose(-1, -2)
    tp = tp.view(Hkv, B, Hq // Hkv, P).transpose(0, 1)
    tp = torch.where(has.unsqueeze(-1), tp, torch.full_like(tp, -math.inf))
    # the sequences' own slots, all of them where a sequence does not have the prefix
    start = torch.where(has, torch.full_like(n, P), torch.zeros_like(n))
    most = int(c["n"])
    slots = (start + torch.arange(most, device="cuda")).expand(B, Hkv, most)
    inside = slots < n
    slots = torch.where(inside, slots, torch.zeros_like(slots))
    own_rows = _rows(s["table"].unsqueeze(1).expand(-1, Hkv, -1), slots, head.view(1, Hkv, 1), Hkv, ps)
    to = q @ kc[own_rows].float().transpose(-1, -2)
    to = torch.where(inside.unsqueeze(2), to, torch.full_like(to, -math.inf))
    m = torch.maximum(tp.amax(-1, keepdim=True), to.amax(-1, keepdim=True))
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    tp, to = torch.exp(tp - m0), torch.exp(to - m0)
    l = tp.sum(-1, keepdim=True) + to.sum(-1, keepdim=True)
    o = (tp.transpose(0, 1).reshape(Hkv, -1, P) @ vc[rows].float()).view(Hkv, B, Hq // Hkv, d).transpose(0, 1)
    o = o + to @ vc[own_rows].float()
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return {"o": o.reshape(B, Hq, d).to(s["q"].dtype), "lse": (m + torch.log(l)).view(B, Hq)}


def _plain_resize(s, lens, new_lens, out):
    ps, table, refs, free = s["case"]["ps"], s["table"], s["refs"], s["free"]
    old, new = (-(-lens.long() // ps)).unsqueeze(1), (-(-new_lens.long() // ps)).unsqueeze(1)
    col = torch.arange(table.shape[1], device="cuda")
    # pages given back, those that nothing else names; the last one goes to the list first
    gone = table[(col >= new) & (col < old)].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    last = torch.zeros_like(refs, dtype=torch.long).scatter_reduce(
        0, gone, torch.arange(1, gone.numel() + 1, device="cuda"), "amax")
    freed = gone[(refs[gone] == 0) & (last[gone] == torch.arange(1, gone.numel() + 1, device="cuda"))]
    at = s["num_free"].long()
    free[at + torch.arange(freed.numel(), device="cuda")] = freed.flip(0).int()
    have = at + freed.numel()
    # pages taken from the list's end, in the order of the sequences, while they last
    need = (new - old).clamp(min=0)
    given = (need.cumsum(0) <= have) | (need == 0)
    fresh = (col >= old) & (col < new) & given
    rank = fresh.flatten().cumsum(0).view(fresh.shape)[fresh]
    pages = free[have - rank]
    table[fresh] = pages
    refs[pages.long()] = 1
    s["num_free"].copy_(have - fresh.sum())
    out.copy_(torch.where(given.squeeze(1), new_lens, lens))


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_bwd"):
        return _exact_rotary(case, s)
    if op == "prefix":
        return _exact_prefix(case, s)
    state = {n: s[n].cpu().numpy().copy() for n in ("table", "refs", "free")}
    state["num_free"] = int(s["num_free"])
    lens, new = _resize_lens(case)
    there = _exact_resize(state, lens, new, case["ps"])
    back = _exact_resize(state, there, lens, case["ps"])
    out = {n: torch.from_numpy(state[n]) for n in ("table", "refs", "free")}
    out["num_free"] = torch.tensor([state["num_free"]], dtype=torch.int32)
    out["there"], out["back"] = torch.tensor(there, dtype=torch.int32), torch.tensor(back, dtype=torch.int32)
    return out


def _exact_rotary(case, s):
    """A pair is a complex number: turning it is a product with amplitude e^(i angle)."""
    N, d, r = case["N"], case["d"], case["r"]
    angle = (s["positions"].double()[:, None] + torch.arange(N, device="cuda").double())[:, :, None] * s["freqs"]
    unit = torch.polar(torch.full_like(angle, s["amplitude"]), angle)  # [B, N, r / 2]
    out = {}
    for name in ("q", "k"):
        x, w = s[name], s[name + "_weight"]
        H = x.shape[1]
        res = torch.empty(x.shape[0], H, N, d, dtype=torch.float64, device="cuda")
        dw = torch.zeros(d, dtype=torch.float64, device="cuda")
        for h in range(H):  # one head at a time
            v = x[:, h].double()
            inv = 1.0 / (v.square().sum(-1, keepdim=True) / d + EPS).sqrt() if w is not None else 1.0
            t = v * inv * w.double() if w is not None else v
            if case["op"] == "rotary_bwd":
                t = s["d" + name][:, h].double()
            turned = t[..., :r]
            pairs = turned.unflatten(-1, (r // 2, 2)) if case["interleaved"] else turned.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_complex(pairs.contiguous()) * (unit.conj() if case["op"] == "rotary_bwd" else unit)
            z = torch.view_as_real(z)
            z = (z if case["interleaved"] else z.transpose(-1, -2)).reshape(turned.shape)
            y = torch.cat([z, t[..., r:]], -1)
            if case["op"] == "rotary_bwd" and w is not None:
                dw += (y * v * inv).sum((0, 1))
                y = y * w.double()
                y = inv * y - v * inv ** 3 * (y * v).sum(-1, keepdim=True) / d
            res[:, h] = y
        out[name] = res
        if case["op"] == "rotary_bwd" and w is not None:
            out[name + "_weight"] = dw
    return out


def _exact_prefix(case, s):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    lens = _own_lens(case)
    P, ps = case["shared"], case["ps"]
    g = Hq // Hkv

    def tokens(cache, pages, lo, hi):  # [Hkv, slots, d]
        first = lo // ps
        t = cache[pages[first:-(-hi // ps)].long()].transpose(0, 1).reshape(Hkv, -1, d)
        return t[:, lo - first * ps:hi - first * ps].double()

    o = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    kp, vp = tokens(s["k_cache"], s["prefix"], 0, P), tokens(s["v_cache"], s["prefix"], 0, P)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        if n >= P:
            k = torch.cat([kp, tokens(s["k_cache"], s["table"][b], P, n)], 1) if n > P else kp
            v = torch.cat([vp, tokens(s["v_cache"], s["table"][b], P, n)], 1) if n > P else vp
        else:
            k, v = tokens(s["k_cache"], s["table"][b], 0, n), tokens(s["v_cache"], s["table"][b], 0, n)
        for h in range(Hkv):
            t = s["q"][b, h * g:(h + 1) * g].double() @ k[h].T / math.sqrt(d)
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(t, -1)
            o[b, h * g:(h + 1) * g] = torch.softmax(t, -1) @ v[h]
    return {"o": o, "lse": lse}


def _exact_resize(state, lens, new, ps):
    table, refs, free = state["table"], state["refs"], state["free"]
    count = lambda n: -(-n // ps)  # noqa: E731
    gone = [int(table[b, i]) for b in range(len(lens)) for i in range(count(new[b]), count(lens[b]))]
    last = {}
    for i, page in enumerate(gone):
        refs[page] -= 1
        last[page] = i
    for i in reversed(range(len(gone))):
        if refs[gone[i]] == 0 and last[gone[i]] == i:
            free[state["num_free"]] = gone[i]
            state["num_free"] += 1
    out, left, ended = [], state["num_free"], False
    for b in range(len(lens)):
        need = max(0, count(new[b]) - count(lens[b]))
        if need > 0 and (ended or need > left):
            ended = True
            out.append(lens[b])
            continue
        for i in range(count(lens[b]), count(lens[b]) + need):
            left -= 1
            table[b, i] = free[left]
            refs[free[left]] = 1
        out.append(new[b])
    state["num_free"] = left
    return out
