"""Drafted tokens and eviction over the paged cache, as cases that can be timed and compared: attention of a tree of
drafted tokens, its verification, the attention weight that cached tokens accumulate, and the eviction of the others.

`own` False computes each operator from elementary torch operations in 32 bits; `own` True calls the library.
Shapes are the ones of this repository's workloads (heads 32/8 of 128, 16/4 of 64, 4/2 of 64).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HELD = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def listed():
    return [
        # a few drafted tokens of one short prompt in single precision: latency
        dict(name="tree-8-over-512", op="tree", B=1, H=4, H_kv=2, d=64, dtype="f32", kind="same", page=16, new_lo=8,
             new_hi=8, kv_lo=512, kv_hi=512, window=0, pad=0, lengths=31),
        # four drafted tokens of each of 16 requests
        dict(name="tree-4-of-16", op="tree", B=16, H=16, H_kv=4, d=64, dtype="bf16", kind="same", page=16, new_lo=4,
             new_hi=4, kv_lo=2048, kv_hi=32768, window=0, pad=8, lengths=32),
        # trees of 20 to 64 drafted tokens of eight requests
        dict(name="tree-64-of-8", op="tree", B=8, H=32, H_kv=8, d=128, dtype="bf16", kind="same", page=64, new_lo=20,
             new_hi=64, kv_lo=4096, kv_hi=32768, window=0, pad=3, lengths=33),
        # one tree over a long prompt in an 8-bit cache
        dict(name="tree-48-over-131072", op="tree", B=1, H=32, H_kv=8, d=128, dtype="bf16", kind="e4m3", page=64,
             new_lo=48, new_hi=48, kv_lo=131072, kv_hi=131072, window=0, pad=0, lengths=34),
        # one decode step of 16 requests adds its weights to the cached tokens'
        dict(name="weights-step-16", op="weights", B=16, H=16, H_kv=4, d=64, dtype="bf16", kind="same", page=16,
             new_lo=1, new_hi=1, kv_lo=2048, kv_hi=32768, window=0, decay=1.0, pad=8, lengths=35),
        # the weights that the last 32 tokens of a long prompt give its tokens, before its cache is cut
        dict(name="weights-last-32-of-131072", op="weights", B=1, H=32, H_kv=8, d=128, dtype="bf16", kind="e4m3",
             page=64, new_lo=32, new_hi=32, kv_lo=131072, kv_hi=131072, window=0, decay=0.0, pad=0, lengths=36),
        # the weights of a whole chunk of a prefill over the chunks before it
        dict(name="weights-chunk-4096", op="weights", B=1, H=32, H_kv=8, d=128, dtype="bf16", kind="same", page=64,
             new_lo=4096, new_hi=4096, kv_lo=32768, kv_hi=32768, window=0, decay=0.875, pad=0, lengths=37),
        # a short prompt's cache cut to 128 tokens in single precision: latency
        dict(name="evict-512-to-128", op="evict", B=1, H_kv=2, d=64, dtype="f32", kind="same", page=16, kv_lo=512,
             kv_hi=512, budget=128, first=4, last=32, shared=False, lengths=38),
        # a long prompt's cache cut to 8192 tokens a head
        dict(name="evict-131072-to-8192", op="evict", B=1, H_kv=8, d=128, dtype="bf16", kind="same", page=64,
             kv_lo=131072, kv_hi=131072, budget=8192, first=4, last=1024, shared=False, lengths=39),
        # 16 requests cut to 2048 tokens, the same ones for every head, in an 8-bit cache that is then read back
        dict(name="evict-batch-16", op="evict", B=16, H_kv=4, d=64, dtype="bf16", kind="int8", page=16, kv_lo=1024,
             kv_hi=32768, budget=2048, first=16, last=256, shared=True, lengths=40),
        # the round of 16 requests with 24 drafted tokens each: their rows into the cache, the walk along the tokens
        # that the target agrees with, and the cache brought in line with it
        dict(name="verify-24-of-16", op="verify", B=16, H_kv=4, d=64, dtype="bf16", kind="same", page=16, new_lo=24,
             new_hi=24, kv_lo=2048, kv_hi=32768, lengths=41),
        # 64 requests with trees of up to 64
        dict(name="verify-64-of-64", op="verify", B=64, H_kv=8, d=128, dtype="bf16", kind="same", page=64, new_lo=9,
             new_hi=64, kv_lo=1024, kv_hi=4096, lengths=42),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "evict", "evict", "verify"])
    H, H_kv, d = rng.choice([(32, 8, 128), (16, 4, 64), (4, 2, 64), (16, 16, 64), (32, 4, 128), (12, 4, 128), (14, 2, 64)])
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    kind = rng.choice(["same", "e4m3", "int8"])
    page = rng.choice([16, 32, 64, 128])
    lengths = rng.randrange(1 << 30)
    B = _spread(rng, 1, 24)
    if op == "verify":
        hi = _spread(rng, 2, 64)
        return dict(op=op, B=B, H_kv=H_kv, d=d, dtype=dtype, kind="same", page=page, new_lo=1, new_hi=hi, kv_lo=hi,
                    kv_hi=_spread(rng, hi, 16384), lengths=lengths)
    if op == "evict":
        kv = _spread(rng, 64, 131072 // B)
        budget = _spread(rng, 32, max(32, min(8192, kv)))
        return dict(op=op, B=B, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, kv_lo=max(1, kv // 16), kv_hi=kv,
                    budget=budget, first=rng.choice([0, 4]), last=rng.randrange(0, budget - 8), shared=rng.random() < 0.4,
                    lengths=lengths)
    window = rng.choice([0, 0, 0, 1000])
    if dtype == "f32":  # the general path: the sizes of the single-precision workload
        H, H_kv, d, B = 4, 2, 64, min(B, 4)
        hi, most = _spread(rng, 1, 32), 2048
    elif op == "tree":
        hi, most = _spread(rng, 1, 128 if B <= 8 else 64), 32768
    else:
        hi, most = (1, 32768) if rng.random() < 0.4 else (_spread(rng, 2, max(2, 2048 // B)), 16384)
    case = dict(op=op, B=B, H=H, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, new_lo=1, new_hi=hi,
                kv_lo=max(hi, 32), kv_hi=_spread(rng, max(hi, 64), most), window=window, pad=rng.choice([0, 0, 5]), lengths=lengths)
    return dict(case, decay=rng.choice([0.0, 1.0, 0.9375])) if op == "weights" else case


def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of each sequence: by the case, the same for every seed."""
    r = np.random.default_rng(case["lengths"])
    kv = r.integers(case["kv_lo"], case["kv_hi"] + 1, case["B"])
    if "new_lo" not in case:
        return np.zeros_like(kv), kv
    new = r.integers(case["new_lo"], case["new_hi"] + 1, case["B"])
    return new, np.maximum(new, kv)


def _parents(r, n):
    """A tree of n drafted tokens: each hangs on the root or, more often, on one of the last few before it."""
    p = np.arange(n) - r.integers(1, 9, n)
    p[r.random(n) < 0.15] = 0
    p = np.maximum(p, 0)
    p[0] = -1
    return p.astype(np.int32)


def _scale_of(x, kind):
    """The power of two that a row of an 8-bit cache is divided by."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    m4, e4 = (0.875, 9) if kind == "e4m3" else (0.9921875, 7)
    return torch.where(top == 0, 1.0, torch.ldexp(torch.ones_like(top), (e - e4 + (m > m4).to(e.dtype)).clamp(min=-100)))


def _codes_of(x, scale, kind):
    y = x / scale[..., None]
    return y.to(torch.float8_e4m3fn) if kind == "e4m3" else y.round().to(torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    up = lambda a, t: torch.from_numpy(np.ascontiguousarray(a).astype(t)).cuda()  # noqa: E731
    d, H_kv, page, B, op, kind = (case[k] for k in ("d", "H_kv", "page", "B", "op", "kind"))
    new, kv = _lengths(case)
    kept = np.minimum(kv, case["budget"]) if op == "evict" else np.zeros_like(kv)
    per, per_to = -(-kv // page), -(-kept // page)
    pages = int(per.sum() + per_to.sum()) + 3
    order, table = r.permutation(pages), np.zeros((B, int(per.max())), np.int32)
    to = np.zeros((B, max(1, int(per_to.max()))), np.int32)  # pages of their own for what is kept
    at = 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        to[b, :per_to[b]] = order[at + per[b]:at + per[b] + per_to[b]]
        at += per[b] + per_to[b]
    T = int(new.sum()) + case.get("pad", 0)
    s = dict(case=case, total=int(new.sum()), T=T, max_new=int(new.max()), max_kv=int(kv.max()),
             cu=up(np.concatenate([[0], np.cumsum(new)]), np.int64), kv=up(kv, np.int64), table=up(table, np.int32))
    for name in ("k", "v"):
        x = torch.randn(pages, H_kv, page, d, generator=g, device="cuda")
        if kind == "same":
            s[name], s[name + "_scale"] = x.to(dt), None
        else:
            x = x.to(dt).float()
            s[name + "_scale"] = _scale_of(x, kind)
            s[name] = _codes_of(x, s[name + "_scale"], kind)
    if op in ("weights", "evict"):  # what tokens have gathered: few hold most of it
        s["weights"] = torch.randn(pages, H_kv, page, generator=g, device="cuda").mul_(1.5).sub_(7).exp_()
    if op in ("tree", "weights"):
        s["q"] = normal(T, case["H"], d)
    if op == "tree":
        s["out"] = torch.zeros(T, case["H"], d, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(case["H"], T, dtype=torch.float32, device="cuda")
    if op in ("tree", "verify"):
        words = -(-s["max_new"] // 32)
        parent = np.concatenate([_parents(r, n) for n in new] + [np.zeros(T - s["total"], np.int32)])
        s["parent"] = up(parent, np.int32)
        s["seen"] = torch.zeros(T, words, dtype=torch.int32, device="cuda")
        s["pos"] = torch.zeros(T, dtype=torch.int32, device="cuda")
    if op == "tree":
        s["seen"][:s["total"]] = _words(_ancestors(s), s)
    if op == "weights":
        # the log-sum-exp of unit normal logits over the tokens that a row sees
        p = np.concatenate([np.arange(c - n, c) for n, c in zip(new, kv)] + [np.ones(case["pad"])])
        p = np.minimum(p + 1, case["window"] or p.max() + 1)
        s["lse"] = torch.log(up(p, np.float32)) + 0.5 + 0.05 * torch.randn(case["H"], T, generator=g, device="cuda")
    if op == "verify":
        s["k_new"], s["v_new"] = normal(T, H_kv, d), normal(T, H_kv, d)
        draft = r.integers(0, 32000, T)
        target = r.integers(0, 32000, T)
        first = np.repeat(np.cumsum(new) - new, new)
        for t in range(T):  # the target agrees with a child of most tokens
            if parent[t] >= 0 and r.random() < 0.5:
                target[first[t] + parent[t]] = draft[t]
        s["draft"], s["target"] = up(draft, np.int32), up(target, np.int32)
        s["path"] = torch.zeros(B, s["max_new"], dtype=torch.int32, device="cuda")
        s["next"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if op == "evict":
        s["to"] = up(to, np.int32)
        s["kept"] = torch.zeros(B, 1 if case["shared"] else H_kv, case["budget"], dtype=torch.int32, device="cuda")
    if op in ("evict", "verify"):
        s["n"] = torch.zeros(B, dtype=torch.int64, device="cuda")
        s["kv_out"] = torch.zeros(B, dtype=torch.int64, device="cuda")
    if op == "evict" and kind != "same":
        s["cu_to"], s["rows_to"] = up(np.concatenate([[0], np.cumsum(kept)]), np.int64), int(kept.sum())
        for name in ("k", "v"):
            s["out_" + name] = torch.zeros(H_kv, s["rows_to"], d, dtype=dt, device="cuda")
    if own:
        import speculative_prefill_token_sp_gb300 as sp
        s["cache"] = sp.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], dtype=dt)
        s["batch"] = sp.Batch(s["cu"], s["kv"], s["table"], rows=T, max_new=s["max_new"])
        if op == "tree":
            size = sp.attend_tree_workspace_size(s["q"], s["cache"], s["batch"])
        elif op == "weights":
            size = sp.attend_weights_workspace_size(s["q"], s["cache"], s["batch"])
        else:
            size = max(sp.sp_cache_workspace_size(), sp.sp_tree_workspace_size())
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        if "cu_to" in s:
            s["batch_to"] = sp.Batch(s["cu_to"], s["kv_out"], s["to"], rows=s["rows_to"], max_new=case["budget"])
    return s


def _read(s, name, page, slot):
    """The rows of these pages and slots as 32-bit values, [..., H_kv, d]."""
    x = s[name][page, :, slot].float()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][page, :, slot][..., None]


def _new(s):
    """Which of [B, max_new] are new tokens, and the parent of each (-1: none)."""
    t = torch.arange(s["max_new"], device="cuda")
    real = t < (s["cu"][1:] - s["cu"][:-1])[:, None]
    row = torch.where(real, s["cu"][:-1, None] + t, 0)
    return real, row, torch.where(real, s["parent"][row].long(), -1)


def _ancestors(s):
    """[B, max_new, max_new]: whether row t is drafted token u, or hangs on it over others."""
    real, _, parent = _new(s)
    n = s["max_new"]
    eye = torch.eye(n, device="cuda")
    step = torch.where(parent >= 0, 1.0, 0.0)[..., None] * eye[parent.clamp(min=0)]
    # I + P + P^2 + ... of a tree, all of its entries 0 or 1
    reach = torch.linalg.solve_triangular(eye - step, eye.expand(step.shape), upper=False, unitriangular=True)
    return (reach > 0.5) & real[..., None]


def _words(reach, s):
    """The rows' bits in words of 32, [total, words]."""
    real, words = _new(s)[0], s["seen"].shape[1]
    bits = torch.nn.functional.pad(reach[real], (0, 32 * words - s["max_new"])).view(-1, words, 32).long()
    value = (bits << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).int()


def _logits(s, scale):
    """Scaled logits [B, H_kv, G, max_new, max_kv], the keys' places in the cache, and which rows are new tokens."""
    case = s["case"]
    H, H_kv, d, page, B = case["H"], case["H_kv"], case["d"], case["page"], case["B"]
    new = s["cu"][1:] - s["cu"][:-1]
    t, i = torch.arange(s["max_new"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    there = i < s["kv"][:, None]
    pages = torch.where(there, s["table"][:, (i // page).clamp(max=s["table"].shape[1] - 1)].long(), 0)
    slot = (i % page).expand(B, -1)
    k = torch.where(there[..., None, None], _read(s, "k", pages, slot), 0.0)
    real = t < new[:, None]
    row = torch.where(real, s["cu"][:-1, None] + t, 0)
    q = s["q"][row].float().view(B, -1, H_kv, H // H_kv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, H_kv, -1, d), k.permute(0, 2, 3, 1)).mul_(scale)
    return x.view(B, H_kv, H // H_kv, s["max_new"], s["max_kv"]), pages, slot, there, real, row


def _tree(s):
    case = s["case"]
    H, H_kv, d, B = case["H"], case["H_kv"], case["d"], case["B"]
    x, pages, slot, there, real, row = _logits(s, 1 / math.sqrt(d))
    v = torch.where(there[..., None, None], _read(s, "v", pages, slot), 0.0)
    new = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(s["max_kv"], device="cuda")
    bits = s["seen"][row]  # [B, max_new, words]
    u = (i - (s["kv"] - new)[:, None])[:, None]  # the new token that a token is, [B, 1, max_kv]
    word = torch.gather(bits, 2, (u // 32).clamp(0, bits.shape[2] - 1).expand(-1, s["max_new"], -1))
    ones = ((bits[..., None] >> torch.arange(32, device="cuda")) & 1).sum((2, 3))
    at = (s["kv"] - new)[:, None] + (ones - 1).clamp(min=0)  # a row's place: behind the cached tokens and those it sees
    seen = torch.where(u < 0, (i > at[..., None] - case["window"]) if case["window"] else True, (word >> (u % 32)) & 1 != 0)
    seen = seen & there[:, None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H_kv, -1, s["max_kv"]), v.permute(0, 2, 1, 3)).view(B, H_kv, H // H_kv, -1, d)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], H, d)
    lse = (m + z.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, s["max_new"], H)
    s["out"][:s["total"]] = o[real].to(s["out"].dtype)
    s["lse"][:, :s["total"]] = lse[real].T
    return s["out"], s["lse"]


def _weights(s):
    case = s["case"]
    x, pages, slot, there, real, row = _logits(s, 1 / math.sqrt(case["d"]))
    B, H_kv, G = x.shape[:3]
    new = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(s["max_kv"], device="cuda")
    at = (s["kv"] - new)[:, None] + torch.arange(s["max_new"], device="cuda")
    seen = (i <= at[..., None]) & real[..., None]
    if case["window"]:
        seen &= i > at[..., None] - case["window"]
    lse = s["lse"].T[row].view(B, -1, H_kv, G).permute(0, 2, 3, 1)
    x = x.sub_(lse[..., None]).exp_().masked_fill_(~seen[:, None, None], 0.0).sum((2, 3))  # [B, H_kv, max_kv]
    old = s["weights"][pages, :, slot].transpose(1, 2) * case["decay"]
    was = i < (s["kv"] - new)[:, None]  # a new token has none yet
    x = x + torch.where(was[:, None] & (case["decay"] > 0), old, 0.0)
    first = (s["kv"] - new - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(new)
    there = there & (i >= first[:, None])
    s["weights"][pages[there], :, slot[there]] = x.transpose(1, 2)[there]
    return s["weights"]


def _evict(s):
    case = s["case"]
    page, budget, H_kv = case["page"], case["budget"], case["H_kv"]
    i, j = torch.arange(s["max_kv"], device="cuda"), torch.arange(budget, device="cuda")
    there = i < s["kv"][:, None]
    pages = torch.where(there, s["table"][:, (i // page).clamp(max=s["table"].shape[1] - 1)].long(), 0)
    w = s["weights"][pages, :, (i % page).expand(case["B"], -1)].transpose(1, 2)
    if case["shared"]:
        w = w.amax(1, keepdim=True)
    w = w.masked_fill(((i < case["first"]) | (i >= s["kv"][:, None] - case["last"]))[:, None], math.inf)
    w = w.masked_fill(~there[:, None], -math.inf)
    n = s["kv"].clamp(max=budget)
    order = w.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    order = torch.where(j < n[:, None, None], order, s["max_kv"]).sort(-1).values
    held = j < n[:, None]
    s["kept"].copy_(torch.where(held[:, None], order, -1))
    s["n"].copy_(n)
    token = torch.where(held[:, None], order, 0).expand(-1, H_kv, -1)
    src_page = torch.gather(s["table"].long()[:, None].expand(-1, H_kv, -1), 2, token // page)[held[:, None].expand_as(token)]
    src_slot = (token % page)[held[:, None].expand_as(token)]
    head = torch.arange(H_kv, device="cuda")[None, :, None].expand_as(token)[held[:, None].expand_as(token)]
    to_page = s["to"].long()[:, (j // page).clamp(max=s["to"].shape[1] - 1)][:, None].expand_as(token)[held[:, None].expand_as(token)]
    to_slot = (j % page).expand_as(token)[held[:, None].expand_as(token)]
    for name in ("k", "v", "k_scale", "v_scale", "weights"):
        x = s[name]
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[to_page, head, to_slot] = x[src_page, head, src_slot]
    s["kv_out"].copy_(n)
    if case["kind"] == "same":
        return s["kept"], s["kv_out"], s["weights"], s["k"], s["v"]
    row = (s["cu_to"][:-1, None, None] + j).expand_as(token)[held[:, None].expand_as(token)]
    for name in ("k", "v"):
        x = s[name][to_page, head, to_slot].float() * s[name + "_scale"][to_page, head, to_slot][:, None]
        s["out_" + name][head, row] = x.to(s["out_" + name].dtype)
    return s["kept"], s["kv_out"], s["weights"], s["out_k"], s["out_v"]


def _verify(s):
    page = s["case"]["page"]
    new = s["cu"][1:] - s["cu"][:-1]
    real, row, parent = _new(s)
    reach, t = _ancestors(s), torch.arange(s["max_new"], device="cuda")
    s["seen"][:s["total"]] = _words(reach, s)
    s["pos"][:s["total"]] = ((s["kv"] - new)[:, None] + reach.sum(-1) - 1)[real].int()
    place = (s["kv"] - new)[:, None] + t
    pg = torch.gather(s["table"].long(), 1, torch.where(real, place // page, 0))
    for name in ("k", "v"):
        s[name][pg[real], :, (place % page)[real]] = s[name + "_new"][:s["total"]]
    # a token goes on from its parent if it is the first of the children that the target agrees with
    agrees = (s["draft"][row] == torch.gather(s["target"][row], 1, parent.clamp(min=0))) & (parent >= 0) & real
    before = (parent[:, :, None] == parent[:, None, :]) & agrees[:, None, :] & (t[None, :] < t[:, None])
    on = (agrees & ~before.any(-1)) | ((t == 0) & real)
    taken = ((reach & ~on[:, None]).sum(-1) == 0) & real
    n = taken.sum(-1)
    path = torch.where(taken, t, s["max_new"]).sort(-1).values
    held = t < n[:, None]
    s["path"].copy_(torch.where(held, path, -1))
    s["n"].copy_(n)
    end = torch.gather(path, 1, (n - 1).clamp(min=0)[:, None])
    s["next"].copy_(torch.where(n > 0, torch.gather(s["target"][row], 1, end.clamp(max=s["max_new"] - 1))[:, 0], -1))
    src = (s["kv"] - new)[:, None] + torch.where(held, path, 0)
    src_page = torch.gather(s["table"].long(), 1, torch.where(held, src // page, 0))[held]
    for name in ("k", "v"):
        s[name][pg[held], :, (place % page)[held]] = s[name][src_page, :, (src % page)[held]]
    s["kv_out"].copy_(s["kv"] - new + n)
    return s["seen"], s["pos"], s["path"], s["n"], s["next"], s["kv_out"], s["k"], s["v"]


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"tree": _tree, "weights": _weights, "evict": _evict, "verify": _verify}[case["op"]](s)
    import speculative_prefill_token_sp_gb300 as sp
    if case["op"] == "tree":
        return sp.attend_tree(s["q"], s["cache"], s["batch"], s["seen"], window=case["window"], out=s["out"],
                              lse=s["lse"], ws=s["ws"])
    if case["op"] == "weights":
        return sp.attend_weights(s["q"], s["cache"], s["batch"], s["lse"], s["weights"], window=case["window"],
                                 decay=case["decay"], ws=s["ws"])
    if case["op"] == "evict":
        sp.cache_choose(s["cache"], s["batch"], s["weights"], case["budget"], first=case["first"], last=case["last"],
                        shared=case["shared"], kept=s["kept"], n_kept=s["n"], ws=s["ws"])
        sp.cache_keep(s["cache"], s["batch"], s["kept"], s["n"], to=s["to"], weights=s["weights"], kv_len=s["kv_out"],
                      ws=s["ws"])
        if case["kind"] == "same":
            return s["kept"], s["kv_out"], s["weights"], s["k"], s["v"]
        sp.cache_read(s["cache"], s["batch_to"], out_k=s["out_k"], out_v=s["out_v"], ws=s["ws"])
        return s["kept"], s["kv_out"], s["weights"], s["out_k"], s["out_v"]
    sp.tree_seen(s["batch"], s["parent"], seen=s["seen"], positions=s["pos"], ws=s["ws"])
    sp.cache_write(s["cache"], s["batch"], s["k_new"], s["v_new"], ws=s["ws"])
    sp.tree_accept(s["batch"], s["parent"], s["draft"], s["target"], path=s["path"], n_path=s["n"], next_token=s["next"],
                   ws=s["ws"])
    sp.cache_keep(s["cache"], s["batch"], s["path"], s["n"], drafted=True, kv_len=s["kv_out"], ws=s["ws"])
    return s["seen"], s["pos"], s["path"], s["n"], s["next"], s["kv_out"], s["k"], s["v"]


def _walk(s, case, seed):
    """Of each sequence: its parents, and every row's drafted tokens from itself to the root."""
    cu, parent = s["cu"].tolist(), s["parent"].tolist()
    for b in range(case["B"]):
        mine = parent[cu[b]:cu[b + 1]]
        lines = []
        for t in range(len(mine)):
            line = [t]
            while mine[line[-1]] >= 0:
                line.append(mine[line[-1]])
            lines.append(line)
        yield b, mine, lines


def _visible(case):
    """How many (query, key) pairs one head sees, and how many keys of the cache any query sees.  A tree's rows see
    about four of its tokens."""
    new, kv = _lengths(case)
    window, pairs, keys = case["window"] or 1 << 30, 0, 0
    for n, c in zip(new.tolist(), kv.tolist()):
        at = np.arange(c - n, c)
        if case["op"] == "tree":
            pairs += n * (min(c - n, window) + min(n, 4))
        else:
            pairs += int(np.minimum(at + 1, window).sum())
        keys += c - max(0, c - n - window + 1)
    return pairs, keys


def work(case):
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    d, H_kv, B = case["d"], case["H_kv"], case["B"]
    held = d * size if case["kind"] == "same" else d + 4  # bytes of one row in the cache
    new, kv = _lengths(case)
    total = int(new.sum())
    if case["op"] in ("tree", "weights"):
        pairs, keys = _visible(case)
        if case["op"] == "tree":
            return {"bytes": total * (case["H"] * (2 * d * size + 4) + 4 * -(-case["new_hi"] // 32)) + 2 * keys * H_kv * held,
                    "flops": 4 * d * case["H"] * pairs}
        old = keys if case["decay"] else 0
        return {"bytes": total * case["H"] * (d * size + 4) + keys * H_kv * (held + 4) + 4 * old * H_kv,
                "flops": 2 * d * case["H"] * pairs}
    if case["op"] == "evict":
        kept = int(np.minimum(kv, case["budget"]).sum())
        read = 0 if case["kind"] == "same" else kept * H_kv * 2 * d * size
        return {"bytes": 4 * int(kv.sum()) * H_kv + 2 * kept * H_kv * (2 * held + 4) + read + 4 * kept * (1 if case["shared"] else H_kv),
                "flops": int(kv.sum()) * H_kv}
    words = -(-case["new_hi"] // 32)
    # the new rows written; four a sequence moved
    moved = 4 * B
    return {"bytes": total * (2 * 2 * H_kv * d * size + 4 * (words + 4)) + moved * 2 * 2 * H_kv * d * size, "flops": total * 8}


def exact(case, seed):
    s = prepare(case, seed)
    new, kv = _lengths(case)
    page, d, H_kv = case["page"], case["d"], case["H_kv"]
    starts = np.concatenate([[0], np.cumsum(new)])

    def places(b, first, last):
        at = torch.arange(first, last, device="cuda")
        return s["table"][b].long()[at // page], at % page

    def rows(name, b, first, last):
        """Rows [first, last) of sequence b, [H_kv, rows, d]."""
        p, slot = places(b, first, last)
        x = s[name].transpose(1, 2)[p, slot].double()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"].transpose(1, 2)[p, slot].double()[..., None]
        return x.transpose(0, 1)

    if case["op"] == "tree":
        out, lse = s["out"].double(), s["lse"].double()
        group = case["H"] // H_kv
        for b, _, lines in _walk(s, case, seed):
            n, c = int(new[b]), int(kv[b])
            k, v = rows("k", b, 0, c), rows("v", b, 0, c)
            unseen = torch.ones(n, c, dtype=torch.bool)
            for t, line in enumerate(lines):
                first = max(0, c - n + len(line) - case["window"]) if case["window"] else 0
                unseen[t, first:c - n] = False
                unseen[t, [c - n + u for u in line]] = False
            unseen = unseen.cuda()
            lo, hi = int(starts[b]), int(starts[b + 1])
            for h in range(case["H"]):
                x = s["q"][lo:hi, h].double() @ k[h // group].T / math.sqrt(d)
                x[unseen] = -math.inf
                z = torch.logsumexp(x, -1)
                out[lo:hi, h] = torch.exp(x - z[:, None]) @ v[h // group]
                lse[h, lo:hi] = z
        return out, lse
    if case["op"] == "weights":
        got = s["weights"].double()
        group = case["H"] // H_kv
        for b in range(case["B"]):
            n, c = int(new[b]), int(kv[b])
            lo, hi = int(starts[b]), int(starts[b + 1])
            first = max(0, c - n - case["window"] + 1) if case["window"] else 0
            k, (p, slot) = rows("k", b, first, c), places(b, first, c)
            at, i = torch.arange(c - n, c, device="cuda")[:, None], torch.arange(first, c, device="cuda")
            unseen = i > at
            if case["window"]:
                unseen |= at - i >= case["window"]
            for h in range(H_kv):
                total = torch.zeros(c - first, dtype=torch.float64, device="cuda")
                for f in range(h * group, (h + 1) * group):
                    x = s["q"][lo:hi, f].double() @ k[h].T / math.sqrt(d) - s["lse"][f, lo:hi].double()[:, None]
                    x[unseen] = -math.inf
                    total += x.exp().sum(0)
                old = got[p, h, slot]
                old[i >= c - n] = 0
                got[p, h, slot] = total + (case["decay"] * old if case["decay"] else 0)
        return got
    if case["op"] == "evict":
        kept, weights = s["kept"].cpu().numpy(), s["weights"].cpu().numpy().astype(np.float64)
        kept[:] = -1
        order, to = s["table"].cpu().numpy(), s["to"].cpu().numpy()
        moved = {name: s[name].double() for name in ("k", "v")} if case["kind"] == "same" else None
        read = None if moved else {name: s["out_" + name].double() for name in ("k", "v")}
        weights_out = weights.copy()
        at = 0
        for b in range(case["B"]):
            c, i = int(kv[b]), np.arange(int(kv[b]))
            n = min(c, case["budget"])
            must = (i < case["first"]) | (i >= c - case["last"])
            mine = weights[order[b, i // page], :, i % page]  # [tokens, H_kv]
            for h in range(H_kv):
                score = mine.max(1) if case["shared"] else mine[:, h]
                best = np.lexsort((i, -score, ~must))[:n]
                best.sort()
                kept[b, 0 if case["shared"] else h, :n] = best
                j = np.arange(n)
                weights_out[to[b, j // page], h, j % page] = weights[order[b, best // page], h, best % page]
                best_t = torch.from_numpy(best).cuda()
                src, dst = s["table"][b].long()[best_t // page], s["to"][b].long()[torch.arange(n, device="cuda") // page]
                for name in ("k", "v"):
                    if moved:
                        moved[name][dst, h, torch.arange(n, device="cuda") % page] = s[name][src, h, best_t % page].double()
                    else:
                        read[name][h, at:at + n] = s[name][src, h, best_t % page].double() * s[name + "_scale"][src, h, best_t % page].double()[:, None]
            at += n
        x = moved or read
        return torch.from_numpy(kept), torch.from_numpy(np.minimum(kv, case["budget"])), torch.from_numpy(weights_out), x["k"], x["v"]
    seen, pos = np.zeros(tuple(s["seen"].shape), np.uint32), np.zeros(s["T"], np.int32)
    path, n_path = np.full((case["B"], s["max_new"]), -1, np.int32), np.zeros(case["B"], np.int64)
    following, kv_out = np.full(case["B"], -1, np.int32), kv.copy()
    draft, target = s["draft"].tolist(), s["target"].tolist()
    held = {name: s[name].double() for name in ("k", "v")}
    for b, mine, lines in _walk(s, case, seed):
        lo, n = int(starts[b]), int(new[b])
        for t, line in enumerate(lines):
            for u in line:
                seen[lo + t, u // 32] |= np.uint32(1 << (u % 32))
            pos[lo + t] = kv[b] - n + len(line) - 1
        taken = [0] if n else []
        while n:
            more = [t for t in range(n) if mine[t] == taken[-1] and draft[lo + t] == target[lo + taken[-1]]]
            if not more:
                break
            taken.append(more[0])
        path[b, :len(taken)], n_path[b], kv_out[b] = taken, len(taken), kv[b] - n + len(taken)
        following[b] = target[lo + taken[-1]] if n else -1
        source = list(range(n))
        source[:len(taken)] = taken
        p, slot = places(b, int(kv[b]) - n, int(kv[b]))
        for name in ("k", "v"):
            held[name].transpose(1, 2)[p, slot] = s[name + "_new"][lo:lo + n].double()[source]
    t = torch.from_numpy
    return t(seen.view(np.int32)), t(pos), t(path), t(n_path), t(following), t(kv_out), held["k"], held["v"]
