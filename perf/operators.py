"""The operators around the scoring path, as cases that can be timed and compared: rotary positions, the paged cache
(written and read back), and the attention of new tokens over it.

`own` False computes each operator from elementary torch operations in 32 bits; `own` True calls the library.
Shapes are the ones of this repository's workloads (heads 32/8 of 128, 16/4 of 64, 4/2 of 64).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def listed():
    return [
        # the queries and keys of one decode step of 16 requests
        dict(name="rotary-step-16", op="rotary", T=16, H=16, H_kv=4, d=64, dtype="bf16", axes=1, interleaved=False,
             last=32768),
        # the kept tokens of a 131072-token prompt, at their original positions
        dict(name="rotary-kept-8192", op="rotary", T=8192, H=32, H_kv=8, d=128, dtype="bf16", axes=1,
             interleaved=False, last=131072),
        # image patches with positions in time, height and width, in single precision
        dict(name="rotary-image-4999", op="rotary", T=4999, H=16, H_kv=4, d=64, dtype="f32", axes=3,
             interleaved=True, last=1500),
        # one decode step's keys and values of 16 requests into an 8-bit cache
        dict(name="store-step-16", op="store", B=16, H_kv=4, d=64, dtype="bf16", kind="int8", page=16,
             new_lo=1, new_hi=1, kv_lo=2048, kv_hi=32768, lengths=11),
        # a prompt's chunk into an 8-bit cache
        dict(name="store-chunk-8192", op="store", B=1, H_kv=8, d=128, dtype="bf16", kind="e4m3", page=64,
             new_lo=8192, new_hi=8192, kv_lo=32768, kv_hi=32768, lengths=12),
        # one layer of a long prompt read back for the scoring call
        dict(name="read-prompt-131072", op="read", B=1, H_kv=8, d=128, dtype="bf16", kind="e4m3", page=64,
             new_lo=131072, new_hi=131072, kv_lo=131072, kv_hi=131072, lengths=13),
        # one layer of 16 prompts read back into the packed layout
        dict(name="read-batch-16", op="read", B=16, H_kv=4, d=64, dtype="bf16", kind="same", page=16,
             new_lo=2048, new_hi=32768, kv_lo=0, kv_hi=0, lengths=14),
        # one token of a short prompt in single precision: latency
        dict(name="attend-token-512", op="attend", B=1, H=4, H_kv=2, d=64, dtype="f32", kind="same", page=16,
             new_lo=1, new_hi=1, kv_lo=512, kv_hi=512, window=0, pad=0, lengths=15),
        # one decode step of 16 requests of 2K to 32K tokens, in a batch padded to 24 rows
        dict(name="attend-step-16", op="attend", B=16, H=16, H_kv=4, d=64, dtype="bf16", kind="same", page=16,
             new_lo=1, new_hi=1, kv_lo=2048, kv_hi=32768, window=0, pad=8, lengths=16),
        # one look-ahead step over a long prompt in an 8-bit cache
        dict(name="attend-step-131072", op="attend", B=1, H=32, H_kv=8, d=128, dtype="bf16", kind="e4m3", page=64,
             new_lo=1, new_hi=1, kv_lo=131072, kv_hi=131072, window=0, pad=0, lengths=17),
        # a chunk of a prefill over the chunks before it
        dict(name="attend-chunk-4096", op="attend", B=1, H=32, H_kv=8, d=128, dtype="bf16", kind="same", page=64,
             new_lo=4096, new_hi=4096, kv_lo=32768, kv_hi=32768, window=0, pad=0, lengths=18),
        # chunks of seven requests at once, of odd lengths, in an 8-bit cache with a sliding window
        dict(name="attend-ragged-7", op="attend", B=7, H=32, H_kv=8, d=128, dtype="bf16", kind="int8", page=32,
             new_lo=1, new_hi=701, kv_lo=701, kv_hi=8191, window=4096, pad=5, lengths=19),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    heads = rng.choice([(32, 8, 128), (16, 4, 64), (4, 2, 64), (16, 16, 64), (32, 4, 128), (12, 4, 128), (14, 2, 64)])
    H, H_kv, d = heads
    op = rng.choice(["rotary", "store", "read", "attend", "attend", "attend"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    kind = rng.choice(["same", "e4m3", "int8"])
    page = rng.choice([16, 32, 64, 128])
    lengths = rng.randrange(1 << 30)
    if op == "rotary":
        return dict(op=op, T=_spread(rng, 1, 8192), H=H, H_kv=H_kv, d=d, dtype=dtype, axes=rng.choice([1, 3]),
                    interleaved=rng.random() < 0.5, last=_spread(rng, 16384, 1 << 20))
    B = _spread(rng, 1, 24)
    if op == "store":
        hi = _spread(rng, 1, max(1, 8192 // B))
        return dict(op=op, B=B, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, new_lo=1, new_hi=hi, kv_lo=hi,
                    kv_hi=_spread(rng, hi, 32768), lengths=lengths)
    if op == "read":
        hi = _spread(rng, 64, 131072 // B)
        return dict(op=op, B=B, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, new_lo=max(1, hi // 16),
                    new_hi=hi, kv_lo=0, kv_hi=0, lengths=lengths)
    if dtype == "f32":  # the general path: the sizes of the single-precision workload
        hi = _spread(rng, 1, 64)
        return dict(op=op, B=min(B, 8), H=4, H_kv=2, d=64, dtype=dtype, kind=kind, page=page, new_lo=1, new_hi=hi,
                    kv_lo=hi, kv_hi=_spread(rng, hi, 2048), window=0, pad=rng.choice([0, 3]), lengths=lengths)
    if rng.random() < 0.5:  # a decode step
        kv = _spread(rng, 64, 32768)
        return dict(op=op, B=B, H=H, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, new_lo=1, new_hi=1,
                    kv_lo=max(1, kv // 16), kv_hi=kv, window=0, pad=rng.choice([0, 0, 8]), lengths=lengths)
    B = min(B, 8)
    hi = _spread(rng, 2, 2048 // B)
    return dict(op=op, B=B, H=H, H_kv=H_kv, d=d, dtype=dtype, kind=kind, page=page, new_lo=1, new_hi=hi, kv_lo=hi,
                kv_hi=_spread(rng, hi, 16384), window=rng.choice([0, 0, 1000]), pad=rng.choice([0, 3]),
                lengths=lengths)


def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of each sequence: by the case, the same for every seed."""
    r = np.random.default_rng(case["lengths"])
    new = r.integers(case["new_lo"], case["new_hi"] + 1, case["B"])
    if not case["kv_hi"]:
        return new, new.copy()
    return new, np.maximum(new, r.integers(case["kv_lo"], case["kv_hi"] + 1, case["B"]))


def _sections(case):
    """How many of the d / 2 pairs each position axis has."""
    pairs = case["d"] // 2
    return (pairs,) if case["axes"] == 1 else (pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8)


def _axis_of_pair(case):
    return [a for a, n in enumerate(_sections(case)) for _ in range(n)]


def _scale_of(x, kind):
    """The power of two that a row of an 8-bit cache is divided by."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    m4, e4 = (0.875, 9) if kind == "e4m3" else (0.9921875, 7)
    k = (e - e4 + (m > m4).to(e.dtype)).clamp(min=-100)
    s = torch.where(top == 0, 1.0, torch.ldexp(torch.ones_like(top), k))
    return torch.where(torch.isfinite(top), s, math.nan)


def _codes_of(x, scale, kind):
    y = torch.where(torch.isnan(scale)[..., None], torch.zeros_like(x), x / scale[..., None])
    return y.to(torch.float8_e4m3fn) if kind == "e4m3" else y.round().to(torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    d, H_kv = case["d"], case["H_kv"]
    if case["op"] == "rotary":
        T = case["T"]
        if case["axes"] == 1:  # ascending positions of kept tokens
            pos = np.sort(r.choice(case["last"], T, replace=False))[None]
        else:  # patches of images: time, height, width
            pos = np.stack([r.integers(0, case["last"], T) for _ in range(case["axes"])])
        s = dict(case=case, q=normal(T, case["H"], d), k=normal(T, H_kv, d),
                 pos=torch.from_numpy(pos.astype(np.int32)).cuda(), base=500000.0)
        if own:
            import speculative_prefill_token_sp_gb300 as sp
            s["plan"] = sp.rotary_plan(d, base=s["base"], sections=_sections(case), interleaved=case["interleaved"])
        return s
    new, kv = _lengths(case)
    page, B = case["page"], case["B"]
    per = -(-kv // page)
    pages = int(per.sum()) + 3
    order, table = r.permutation(pages), np.zeros((B, int(per.max())), np.int32)
    for b, first in enumerate(np.cumsum(per) - per):
        table[b, :per[b]] = order[first:first + per[b]]
    T = int(new.sum()) + case.get("pad", 0)
    s = dict(case=case, total=int(new.sum()), T=T, max_new=int(new.max()), max_kv=int(kv.max()),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int64)).cuda(),
             kv=torch.from_numpy(kv.astype(np.int64)).cuda(), table=torch.from_numpy(table).cuda())
    kind = case["kind"]
    for name in ("k", "v"):
        x = torch.randn(pages, H_kv, page, d, generator=g, device="cuda")
        if kind == "same":
            s[name], s[name + "_scale"] = x.to(dt), None
        else:
            x = x.to(dt).float()
            s[name + "_scale"] = _scale_of(x, kind)
            s[name] = _codes_of(x, s[name + "_scale"], kind)
    if case["op"] == "store":
        s["k_new"], s["v_new"] = normal(T, H_kv, d), normal(T, H_kv, d)
    if case["op"] in ("store", "read"):
        s["out_k"] = torch.zeros(H_kv, T, d, dtype=dt, device="cuda")
        s["out_v"] = torch.zeros(H_kv, T, d, dtype=dt, device="cuda")
    if case["op"] == "attend":
        s["q"] = normal(T, case["H"], d)
        s["out"] = torch.zeros(T, case["H"], d, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(case["H"], T, dtype=torch.float32, device="cuda")
    if own:
        import speculative_prefill_token_sp_gb300 as sp
        s["cache"] = sp.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], dtype=dt)
        s["batch"] = sp.Batch(s["cu"], s["kv"], s["table"], rows=T, max_new=s["max_new"])
        if case["op"] == "attend":
            s["ws"] = torch.empty(sp.attend_workspace_size(s["q"], s["cache"], s["batch"]), dtype=torch.uint8,
                                  device="cuda")
        else:
            s["ws"] = torch.empty(sp.sp_cache_workspace_size(), dtype=torch.uint8, device="cuda")
    return s


def _rotary(x, pos, case, base):
    pairs = case["d"] // 2
    freq = base ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    axis = torch.tensor(_axis_of_pair(case), device="cuda")
    angle = pos[axis].double().T * freq  # [T, pairs], in 64 bits: positions reach 10^6
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2).to(x.dtype)
    a, b = y[..., :pairs], y[..., pairs:]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


def _places(s):
    """(page, slot) in the cache of each new token."""
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:], t, right=True)
    at = s["kv"][b] - s["cu"][b + 1] + t
    page = s["case"]["page"]
    return s["table"][b, at // page].long(), at % page


def _read(s, name, page, slot):
    """The rows of these pages and slots as 32-bit values, [..., H_kv, d]."""
    x = s[name][page, :, slot].float()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][page, :, slot][..., None]


def _attend(s):
    case = s["case"]
    H, H_kv, d, page, B = case["H"], case["H_kv"], case["d"], case["page"], case["B"]
    new = s["cu"][1:] - s["cu"][:-1]
    t, i = torch.arange(s["max_new"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    there = i < s["kv"][:, None]  # [B, max_kv]
    pages = torch.where(there, s["table"][:, i // page].long(), 0)
    slot = (i % page).expand(B, -1)
    k = torch.where(there[..., None, None], _read(s, "k", pages, slot), 0.0)
    v = torch.where(there[..., None, None], _read(s, "v", pages, slot), 0.0)
    row = torch.where(t < new[:, None], s["cu"][:-1, None] + t, 0)
    q = s["q"][row].float().view(B, -1, H_kv, H // H_kv, d).permute(0, 2, 3, 1, 4)  # [B, H_kv, G, max_new, d]
    x = torch.matmul(q.reshape(B, H_kv, -1, d), k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
    x = x.view(B, H_kv, H // H_kv, s["max_new"], s["max_kv"])
    at = (s["kv"] - new)[:, None] + t
    seen = (i <= at[..., None]) & there[:, None]
    if case["window"]:
        seen &= i > at[..., None] - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H_kv, -1, s["max_kv"]), v.permute(0, 2, 1, 3)).view(q.shape)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], H, d)
    lse = (m + z.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, s["max_new"], H)
    real = t < new[:, None]
    s["out"][:s["total"]] = o[real].to(s["out"].dtype)
    s["lse"][:, :s["total"]] = lse[real].T
    return s["out"], s["lse"]


def run(state):
    s, case = state, state["case"]
    if own:
        import speculative_prefill_token_sp_gb300 as sp
        if case["op"] == "rotary":
            return sp.rotary(s["q"], s["k"], s["pos"], s["plan"])
        if case["op"] == "attend":
            return sp.attend(s["q"], s["cache"], s["batch"], window=case["window"], out=s["out"], lse=s["lse"],
                             ws=s["ws"])
        if case["op"] == "store":
            sp.cache_write(s["cache"], s["batch"], s["k_new"], s["v_new"], ws=s["ws"])
        return sp.cache_read(s["cache"], s["batch"], out_k=s["out_k"], out_v=s["out_v"], ws=s["ws"])
    if case["op"] == "rotary":
        return _rotary(s["q"], s["pos"], case, s["base"]), _rotary(s["k"], s["pos"], case, s["base"])
    if case["op"] == "attend":
        return _attend(s)
    page, slot = _places(s)
    if case["op"] == "store":
        for name in ("k", "v"):
            x = s[name + "_new"][:s["total"]]
            if case["kind"] == "same":
                s[name][page, :, slot] = x
            else:
                scale = _scale_of(x.float(), case["kind"])
                codes = _codes_of(x.float(), scale, case["kind"])
                s[name].view(torch.int8)[page, :, slot] = codes.view(torch.int8)
                s[name + "_scale"][page, :, slot] = scale
    for name in ("k", "v"):
        s["out_" + name][:, :s["total"]] = _read(s, name, page, slot).transpose(0, 1).to(s["out_" + name].dtype)
    return s["out_k"], s["out_v"]


def _visible(case):
    """How many (query, key) pairs one head sees, and how many keys of the cache any query sees."""
    new, kv = _lengths(case)
    pairs = keys = 0
    for n, c in zip(new.tolist(), kv.tolist()):
        at = np.arange(c - n, c)
        first = np.maximum(0, at - case["window"] + 1) if case["window"] else np.zeros_like(at)
        pairs += int((at - first + 1).sum())
        keys += c - int(first.min())
    return pairs, keys


def work(case):
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    d, H_kv = case["d"], case["H_kv"]
    if case["op"] == "rotary":
        rows = case["T"] * (case["H"] + H_kv)
        return {"bytes": 2 * rows * d * size + 4 * case["axes"] * case["T"], "flops": 3 * rows * d}
    held = d * size if case["kind"] == "same" else d + 4  # bytes of one row in the cache
    total = int(_lengths(case)[0].sum())
    if case["op"] == "attend":
        pairs, keys = _visible(case)
        return {"bytes": 2 * total * case["H"] * d * size + 4 * total * case["H"] + 2 * keys * H_kv * held,
                "flops": 4 * d * case["H"] * pairs}
    rows = 2 * total * H_kv
    if case["op"] == "store":
        return {"bytes": rows * (2 * d * size + held), "flops": 2 * rows * d}
    return {"bytes": rows * (d * size + held), "flops": rows * d}


def _exact_rotary(case, s, x):
    x = x.double().cpu().numpy()
    pos = s["pos"].cpu().numpy().astype(np.float64)
    pairs = case["d"] // 2
    out = np.empty_like(x)
    for i, axis in enumerate(_axis_of_pair(case)):
        angle = (pos[axis] * s["base"] ** (-i / pairs))[:, None]
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
        out[..., a] = x[..., a] * np.cos(angle) - x[..., b] * np.sin(angle)
        out[..., b] = x[..., b] * np.cos(angle) + x[..., a] * np.sin(angle)
    return out


def _exact_rows(case, x):
    """What rows come back as from an 8-bit cache, in 64 bits."""
    if case["kind"] == "same":
        return x
    top = x.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(top / LARGEST[case["kind"]])).clamp(min=-100)
    k = k + (top > LARGEST[case["kind"]] * torch.exp2(k)).double() - (top <= LARGEST[case["kind"]] * torch.exp2(k - 1)).double()
    s = torch.exp2(torch.where(top > 0, k.clamp(min=-100), 0.0))
    y = x / s
    if case["kind"] == "int8":
        return y.round() * s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step * s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s, s["q"]), _exact_rotary(case, s, s["k"])
    new, kv = _lengths(case)
    page, d, H_kv = case["page"], case["d"], case["H_kv"]

    def rows(name, b, first, last):
        """Rows [first, last) of sequence b, [H_kv, rows, d]."""
        at = torch.arange(first, last, device="cuda")
        p = s["table"][b].long()[at // page]
        x = s[name].transpose(1, 2)[p, at % page].double()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"].transpose(1, 2)[p, at % page].double()[..., None]
        return x.transpose(0, 1)

    starts = np.concatenate([[0], np.cumsum(new)])
    if case["op"] != "attend":
        got = []
        for name in ("k", "v"):
            out = s["out_" + name].double()
            for b in range(case["B"]):
                lo, hi = int(starts[b]), int(starts[b + 1])
                if case["op"] == "store":
                    out[:, lo:hi] = _exact_rows(case, s[name + "_new"][lo:hi].double()).transpose(0, 1)
                else:
                    out[:, lo:hi] = rows(name, b, int(kv[b] - new[b]), int(kv[b]))
            got.append(out)
        return tuple(got)
    out, lse = s["out"].double(), s["lse"].double()
    group = case["H"] // H_kv
    for b in range(case["B"]):
        n, c = int(new[b]), int(kv[b])
        k, v = rows("k", b, 0, c), rows("v", b, 0, c)
        at = torch.arange(c - n, c, device="cuda")[:, None]
        i = torch.arange(c, device="cuda")
        unseen = i > at
        if case["window"]:
            unseen |= at - i >= case["window"]
        for h in range(case["H"]):
            x = s["q"][int(starts[b]):int(starts[b + 1]), h].double() @ k[h // group].T / math.sqrt(d)
            x[unseen] = -math.inf
            z = torch.logsumexp(x, -1)
            out[int(starts[b]):int(starts[b + 1]), h] = torch.exp(x - z[:, None]) @ v[h // group]
            lse[h, int(starts[b]):int(starts[b + 1])] = z
    return out, lse
