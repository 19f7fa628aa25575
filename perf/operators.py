"""What the operators around the block-sparse self-attention of a video diffusion
transformer are measured on: attention of the video tokens to an encoder's states of another
length (forward, and forward with its gradients), and layer norm (forward, and forward with
its gradients).

Where `own` is false, run() computes the plain form, elementary torch operations in fp32
rounded once at the end; where it is true, it calls the library.

    cross attention  out = softmax(scale q k^T) v over the valid keys of the batch item,
                     lse = the natural log of the sum of exponentials; query head h reads
                     key head h // (H / Hkv); an item without a valid key gives 0 and -inf
    layer norm       y = (x - mean) rstd (offset + weight) + bias over the last axis,
                     rstd = 1 / sqrt(var + eps); weight and bias are absent, one for all rows
                     or one per batch item (the modulation of a diffusion transformer, whose
                     weight is the distance from one)
"""
import math

import torch

own = False

EPS = 1e-6


def _attn(name, B, N, M, H, Hkv, d, pad, train):
    return {"name": name, "op": "cross_attn", "B": B, "N": N, "M": M, "H": H, "Hkv": Hkv, "d": d, "pad": pad,
            "train": train}


def _norm(name, B, N, C, x, y, affine, train):
    return {"name": name, "op": "layer_norm", "B": B, "N": N, "C": C, "x": x, "y": y, "affine": affine,
            "train": train}


def listed():
    return [
        # one query token (a pooled token, or the first step of a streamed clip): latency
        _attn("attn_one_query", 1, 1, 512, 12, 12, 128, "none", False),
        # a few learned queries that summarise a long encoding, shared key heads, ragged
        _attn("attn_few_queries_long_encoder", 2, 16, 32768, 24, 8, 128, "len", False),
        # a small batch of clips with prompts of any length, one of them empty; odd sizes
        _attn("attn_ragged_d64", 3, 1001, 77, 10, 2, 64, "len", False),
        # the 40-head 21 x 45 x 80 call attending to a prompt padded to 512 tokens
        _attn("attn_wan14b_prompt512", 1, 75600, 512, 40, 40, 128, "none", False),
        # the 24-head 33 x 45 x 80 call with a padding mask over 256 prompt tokens
        _attn("attn_hunyuan_prompt256", 1, 118800, 256, 24, 24, 128, "mask", False),
        # training steps: the 12-head 21 x 30 x 52 call; shared key heads, odd sizes, a mask
        _attn("attn_train_wan13b_prompt512", 1, 32760, 512, 12, 12, 128, "none", True),
        _attn("attn_train_ragged_d64", 4, 1237, 333, 8, 2, 64, "mask", True),
        # one token of a 12 x 128 wide model: latency
        _norm("norm_one_token", 1, 1, 1536, "bf16", "bf16", "item", False),
        # queries normalised per head ahead of attention
        _norm("norm_per_head_wan13b", 1, 32760 * 12, 128, "bf16", "bf16", "shared", False),
        # the modulated norm ahead of each part of a block, 40 x 128 wide
        _norm("norm_wan14b", 1, 75600, 5120, "bf16", "bf16", "item", False),
        # training: residual stream in fp32, modulated per clip; and an odd width
        _norm("norm_train_wan13b_fp32", 2, 32760, 1536, "fp32", "bf16", "item", True),
        _norm("norm_train_odd", 1, 4099, 1001, "bf16", "bf16", "shared", True),
    ]


# a drawn case does at most the work of the largest listed one of its operator
_MOST_FLOPS = 4.0 * 75600 * 512 * 40 * 128
_MOST_ELEMENTS = 75600 * 5120


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    train = rng.random() < 0.4
    if rng.random() < 0.5:
        B = rng.choice([1, 1, 2, 3, 4])
        H, Hkv = rng.choice([(2, 2), (12, 12), (24, 24), (40, 40), (24, 8), (10, 2), (8, 1), (6, 2)])
        d = rng.choice([64, 128, 128])
        N = _log_int(rng, 1, 118800)
        M = _log_int(rng, 1, 32768 if N <= 64 else 2048)
        per = 4.0 * B * H * d * (3.5 if train else 1.0)
        if per * N * M > _MOST_FLOPS:
            N = max(1, int(_MOST_FLOPS / (per * M)))
        return _attn("", B, N, M, H, Hkv, d, rng.choice(["none", "len", "mask"]), train) | {"name": "drawn"}
    B = rng.choice([1, 1, 2, 3, 5])
    C = rng.choice([64, 128, 1536, 5120, _log_int(rng, 32, 8192), 8 * _log_int(rng, 4, 1024)])
    N = _log_int(rng, 1, 393120)
    most = _MOST_ELEMENTS // (3 if train else 1)
    N = max(1, min(N, most // (B * C)))
    x = rng.choice(["bf16", "bf16", "fp32"])
    y = "bf16" if x == "bf16" else rng.choice(["bf16", "fp32"])
    return _norm("drawn", B, N, C, x, y, rng.choice(["none", "shared", "item"]), train)


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _valid_keys(case, gen):
    """(kv_len int32 [B] or None, key_mask bool [B, M] or None)."""
    B, M = case["B"], case["M"]
    if case["pad"] == "len":
        n = torch.randint(1, M + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        if B > 2:
            n[1] = 0                     # an empty prompt in the batch
        return n, None
    if case["pad"] == "mask":
        m = torch.rand((B, M), generator=gen, device="cuda") < 0.8
        if B > 2:
            m[1] = False
        return None, m
    return None, None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def rand(shape, dtype):
        # drawn in pieces, so that the fp32 draw of a large tensor does not stand beside it
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat = out.view(-1)
        for at in range(0, flat.numel(), 1 << 28):
            part = flat[at:at + (1 << 28)]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
        return out

    s = dict(case)
    B, N = case["B"], case["N"]
    if case["op"] == "cross_attn":
        M, H, Hkv, d = case["M"], case["H"], case["Hkv"], case["d"]
        s["q"] = rand((B, N, H, d), torch.bfloat16)
        s["k"] = rand((B, M, Hkv, d), torch.bfloat16)
        s["v"] = rand((B, M, Hkv, d), torch.bfloat16)
        s["kv_len"], s["key_mask"] = _valid_keys(case, gen)
        if case["train"]:
            s["dout"] = rand((B, N, H, d), torch.bfloat16)
        if own:
            import block_sparse_attention_major_b200 as bsa
            s["geometry"] = bsa.CrossGeometry(B, H, Hkv, d, N, M)
            s["ws"] = bsa.alloc_cross_workspace(s["geometry"])
    else:
        C = case["C"]
        s["x"] = rand((B, N, C), _TYPES[case["x"]])
        # rows as a residual stream has them: away from zero, each row at a level and a scale of its own
        s["x"].mul_(0.25 + 4.0 * torch.rand((B, N, 1), generator=gen, device="cuda"))
        s["x"].add_(torch.randn((B, N, 1), generator=gen, device="cuda"))
        s["weight"] = s["bias"] = None
        s["offset"] = 0.0
        if case["affine"] == "shared":
            s["weight"] = 1.0 + 0.1 * rand((C,), torch.float32)
            s["bias"] = 0.1 * rand((C,), torch.float32)
        elif case["affine"] == "item":
            s["weight"] = 0.2 * rand((B, C), torch.float32)
            s["bias"] = 0.2 * rand((B, C), torch.float32)
            s["offset"] = 1.0
        if case["train"]:
            s["dy"] = rand((B, N, C), _TYPES[case["y"]])
            if own:
                import block_sparse_attention_major_b200 as bsa
                s["ws"] = bsa.alloc_layer_norm_workspace(s["x"], s["weight"])
    return s


def _run_own(s):
    import block_sparse_attention_major_b200 as bsa
    if s["op"] == "cross_attn":
        pad = dict(kv_len=s["kv_len"], key_mask=s["key_mask"], ws=s["ws"])
        out, lse = bsa.cross_attn_fwd(s["geometry"], s["q"], s["k"], s["v"], **pad)
        if not s["train"]:
            return {"out": out, "lse": lse}
        dq, dk, dv = bsa.cross_attn_bwd(s["geometry"], s["q"], s["k"], s["v"], out, lse, s["dout"], **pad)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    y, mean, rstd = bsa.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS, weight_offset=s["offset"],
                                       out_dtype=_TYPES[s["y"]])
    if not s["train"]:
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = bsa.layer_norm_bwd(s["x"], s["dy"], mean, rstd, s["weight"], weight_offset=s["offset"],
                                    want_bias=s["bias"] is not None, ws=s["ws"])
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx} | ({} if dw is None else {"dweight": dw, "dbias": db})


def _valid(kv_len, key_mask, M):
    """bool [B, 1, 1, 1, M], or None where every key is valid."""
    if kv_len is not None:
        ok = torch.arange(M, device=kv_len.device)[None] < kv_len[:, None]
    elif key_mask is not None:
        ok = key_mask
    else:
        return None
    return ok[:, None, None, None]


def _plain_attn(s):
    B, N, H, d = s["q"].shape
    M, Hkv = s["k"].shape[1:3]
    G, scale = H // Hkv, 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4)              # [B, Hkv, G, N, d]
    k, v = (s[n].float().permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))    # [B, Hkv, 1, M, d]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    ok = _valid(s["kv_len"], s["key_mask"], M)
    if ok is not None:
        p.masked_fill_(~ok, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)              # rows without a key
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    out = torch.matmul(p, v)

    def heads(x):                                                                # -> [B, N, H, d]
        return x.permute(0, 3, 1, 2, 4).reshape(B, N, H, d).to(torch.bfloat16)

    r = {"out": heads(out), "lse": (top + total.log()).reshape(B, H, N)}
    if not s["train"]:
        return r
    g = s["dout"].float().view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), g).sum(2)                             # [B, Hkv, M, d]
    ds = torch.matmul(g, v.transpose(-1, -2))
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    r["dq"] = heads(torch.matmul(ds, k))
    r["dk"] = torch.matmul(ds.transpose(-1, -2), q).sum(2).transpose(1, 2).to(torch.bfloat16)
    r["dv"] = dv.transpose(1, 2).to(torch.bfloat16)
    return r


def _plain_norm(s):
    x = s["x"].float()
    C = x.shape[-1]
    mean = x.sum(-1, keepdim=True) / C
    xhat = x - mean
    rstd = 1.0 / torch.sqrt((xhat * xhat).sum(-1, keepdim=True) / C + EPS)
    xhat.mul_(rstd)
    w = s["weight"]
    if w is not None:
        w = (w + s["offset"]).view(-1, 1, C)
        y = xhat * w + s["bias"].view(-1, 1, C)
    else:
        y = xhat
    r = {"y": y.to(_TYPES[s["y"]]), "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if not s["train"]:
        return r
    dy = s["dy"].float()
    g = dy if w is None else dy * w
    dx = g - g.sum(-1, keepdim=True) / C
    dx -= xhat * ((g * xhat).sum(-1, keepdim=True) / C)
    r["dx"] = dx.mul_(rstd).to(s["x"].dtype)
    if w is not None:
        # sums over up to 393120 rows: in 64 bits
        over = (1,) if s["affine"] == "item" else (0, 1)
        r["dweight"] = (dy * xhat).sum(over, dtype=torch.float64).float()
        r["dbias"] = dy.sum(over, dtype=torch.float64).float()
    return r


def run(state):
    if own:
        return _run_own(state)
    return _plain_attn(state) if state["op"] == "cross_attn" else _plain_norm(state)


def work(case):
    B, N = case["B"], case["N"]
    if case["op"] == "cross_attn":
        M, H, Hkv, d = case["M"], case["H"], case["Hkv"], case["d"]
        q, kv, lse = 2.0 * B * N * H * d, 2.0 * B * M * Hkv * d, 4.0 * B * N * H
        bytes_ = 2 * q + 2 * kv + lse
        flops = 4.0 * B * N * M * H * d
        if case["train"]:
            bytes_ += 2 * q + 2 * kv
            flops *= 3.5
        return {"bytes": bytes_, "flops": flops}
    size = {"bf16": 2, "fp32": 4}
    n, C = float(B * N), case["C"]
    affine = {"none": 0, "shared": 1, "item": B}[case["affine"]] * 8.0 * C
    bytes_ = n * C * (size[case["x"]] + size[case["y"]]) + 8.0 * n + affine
    flops = 8.0 * n * C
    if case["train"]:
        bytes_ += n * C * (size[case["x"]] + size[case["y"]]) + affine
        flops += 14.0 * n * C
    return {"bytes": bytes_, "flops": flops}


def _exact_attn(case, s):
    """Key by key in the definition's order: weights exp(s - lse), then the sums, per head."""
    B, N, M, H, Hkv, d = (case[n] for n in ("B", "N", "M", "H", "Hkv", "d"))
    f8 = torch.float64
    out = torch.zeros((B, N, H, d), dtype=f8, device="cuda")
    lse = torch.full((B, H, N), -math.inf, dtype=f8, device="cuda")
    train = case["train"]
    dq = torch.zeros_like(out) if train else None
    dk = torch.zeros((B, M, Hkv, d), dtype=f8, device="cuda") if train else None
    dv = torch.zeros_like(dk) if train else None
    step = max(1, (1 << 27) // M)
    for b in range(B):
        keys = torch.arange(M, device="cuda")
        if s["kv_len"] is not None:
            keys = keys[: int(s["kv_len"][b])]
        elif s["key_mask"] is not None:
            keys = keys[s["key_mask"][b]]
        if keys.numel() == 0:
            continue
        for h in range(H):
            c = h * Hkv // H
            kk, vv = s["k"][b, keys, c].to(f8), s["v"][b, keys, c].to(f8)
            for at in range(0, N, step):
                part = slice(at, min(N, at + step))
                qq = s["q"][b, part, h].to(f8) / math.sqrt(d)
                z = qq @ kk.T
                l = torch.logsumexp(z, 1)
                w = torch.exp(z - l[:, None])
                o = w @ vv
                out[b, part, h], lse[b, h, part] = o, l
                if train:
                    g = s["dout"][b, part, h].to(f8)
                    t = w * (g @ vv.T)
                    t -= w * t.sum(1, keepdim=True)
                    dq[b, part, h] = (t @ kk) / math.sqrt(d)
                    dk[b, :, c].index_add_(0, keys, t.T @ qq)
                    dv[b, :, c].index_add_(0, keys, w.T @ g)
    r = {"out": out, "lse": lse}
    return r | {"dq": dq, "dk": dk, "dv": dv} if train else r


def _exact_norm(case, s):
    B, N, C = case["B"], case["N"], case["C"]
    f8 = torch.float64
    y = torch.empty((B, N, C), dtype=f8, device="cuda")
    mean = torch.empty((B, N), dtype=f8, device="cuda")
    rstd = torch.empty_like(mean)
    train, affine = case["train"], case["affine"] != "none"
    dx = torch.empty_like(y) if train else None
    groups = B if case["affine"] == "item" else 1
    dw, db = (torch.zeros((groups, C), dtype=f8, device="cuda") for _ in range(2))
    step = max(1, (1 << 26) // C)
    for b in range(B):
        i = b if groups > 1 else 0
        w = s["weight"].view(groups, C)[i].to(f8) + s["offset"] if affine else torch.ones(C, dtype=f8, device="cuda")
        for at in range(0, N, step):
            part = slice(at, min(N, at + step))
            x = s["x"][b, part].to(f8)
            var, mu = torch.var_mean(x, 1, correction=0)
            inv = (var + EPS).rsqrt()
            n = (x - mu[:, None]) * inv[:, None]
            y[b, part] = n * w + s["bias"].view(groups, C)[i].to(f8) if affine else n
            mean[b, part], rstd[b, part] = mu, inv
            if train:
                g = s["dy"][b, part].to(f8)
                dw[i] += (g * n).sum(0)
                db[i] += g.sum(0)
                t = g * w
                dx[b, part] = inv[:, None] * (t - t.mean(1, keepdim=True) - n * (t * n).mean(1, keepdim=True))
    r = {"y": y, "mean": mean, "rstd": rstd}
    if train:
        r["dx"] = dx
        if affine:
            r["dweight"], r["dbias"] = (dw, db) if case["affine"] == "item" else (dw[0], db[0])
    return r


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"] == "cross_attn" else _exact_norm(case, s)
