"""Shared by the tests of the paged cache and the attention over it: random caches and batches, and error bounds."""
import numpy as np


def make_cache(sp, rng, *, H_kv, d, page, kv, kind="same", dtype=None, layout="hnd", spare=2, junk=None, device="cuda"):
    """A cache that holds sequences of lengths kv, with shuffled pages.  Returns (Cache, table int32 [B, width],
    keys, values): per sequence the values held, float64 [H_kv, kv[b], d].  Unwritten slots hold `junk`."""
    import torch

    import oracle
    dtype = dtype or torch.bfloat16
    B = len(kv)
    per = [-(-n // page) for n in kv]
    pages = sum(per) + spare
    order = rng.permutation(pages)
    width = max(max(per), 1)
    table = np.full((B, width), -7, dtype=np.int32)             # entries past a sequence's pages are never read
    at = 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    held = {"same": dtype, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[kind]
    shape = (pages, H_kv, page, d)

    def side():
        x = torch.from_numpy(rng.standard_normal(shape)).to(dtype).double().numpy()
        if kind == "same":
            full, scale = torch.from_numpy(x).to(dtype), None
            if junk is not None:
                full = full.float()
        else:
            codes, s = oracle.paged.quantise(x, kind)
            x = codes * s[..., None]
            full = torch.from_numpy(codes).to(torch.float32)
            scale = torch.from_numpy(s).float()
        used = np.zeros((pages, page), dtype=bool)
        for b in range(B):
            for i in range(kv[b]):
                used[table[b, i // page], i % page] = True
        unused = torch.from_numpy(~used)[:, None, :].expand(pages, H_kv, page)
        if junk is not None:
            if kind == "int8":
                scale[unused] = float("nan")
            else:
                full = full.float()
                full[unused] = junk
                if scale is not None:
                    scale[unused] = float("nan")
        full = full.to(held) if kind != "int8" else full.to(torch.int8)
        if layout == "nhd":         # [pages, page, H_kv, d], seen as [pages, H_kv, page, d]
            raw = full.view(torch.uint8 if kind != "same" else full.dtype).permute(0, 2, 1, 3).contiguous().to(device)
            full = raw.permute(0, 2, 1, 3).view(held) if kind == "same" else raw.view(held).permute(0, 2, 1, 3)
        else:
            full = full.to(device)
        values = [np.stack([x[table[b, i // page], :, i % page] for i in range(kv[b])], 1) if kv[b] else
                  np.zeros((H_kv, 0, d)) for b in range(B)]
        return full, None if scale is None else scale.to(device), values

    k, ks, kval = side()
    v, vs, vval = side()
    return sp.Cache(k, v, ks, vs, dtype=dtype), table, kval, vval


def make_batch(sp, new, kv, table, *, rows=None, max_new=None, first=0, device="cuda"):
    import torch
    cu = np.concatenate([[first], first + np.cumsum(new)]).astype(np.int64)
    rows = int(cu[-1]) if rows is None else rows
    table = np.where(table < 0, 0x7ffffff0, table)              # a page index that must not be followed
    return sp.Batch(torch.from_numpy(cu).to(device), torch.tensor(kv, dtype=torch.int64, device=device),
                    torch.from_numpy(table.astype(np.int32)).to(device), rows=rows, max_new=max_new), cu


def attend_bounds(dtype, d, keys, ref, spread, top, lse):
    """Error bounds of the attention's out and lse for one sequence.

    A logit is a sum of d products of the inputs, each product and each addition off by at most 2^-24 of the sum of
    magnitudes (`top`), times the scale (two more roundings); in base 2 exponentials add 2^-22 and the conversion
    of the exponent's argument 2^-23 of its magnitude: dx = (d + 6) 2^-24 top + 2^-21 in all.  A weight is then off by
    a factor of e^(2 dx) (its own and the normaliser's), sums of `keys` terms by keys * 2^-24 (in any order, the sums
    rescaled no more often than there are keys: twice that), and bf16 weights by 2^-8.  The result is rounded once:
    2^-8 (bf16) or 2^-24 of it."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    dx = (d + 6) * 2.0 ** -24 * top + 2.0 ** -21
    weight = np.expm1(2 * dx) + 3 * keys * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    out = weight[..., None] * spread * (1 + half) + half * np.abs(ref) + 1e-30
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return out, dx.T + keys * 2.0 ** -23 + 2.0 ** -22 * (1 + finite)
