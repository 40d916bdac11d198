"""The transformer-block operators of the voxel models, as cases that can be timed and checked.

Three operators work next to the convolution on the same rows (one row per active voxel):

* layer normalisation of the feature rows, and its backward pass;
* the rotation of query and key heads by the voxel's coordinates (several axes), and its inverse,
  which is its gradient;
* softmax attention inside each entry of a ragged batch, and its backward pass.

`run` computes a case either through the package (`own` true) or in a plain form made of elementary
torch operations in 32 bits; `exact` computes the same in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
_TYPES = {F32: torch.float32, BF16: torch.bfloat16}


def listed():
    return [
        # one training step's norm on the smallest voxel set (16^3 sphere): latency
        dict(name="norm_train_450x16_f32", op="norm_train", rows=450, channels=16, dtype=F32, params=F32),
        # inference norm on the rows of a batch of four 256^3 sets at 64 channels
        dict(name="norm_1187k_x64_bf16", op="norm", rows=1187403, channels=64, dtype=BF16, params=BF16),
        # training norm of a wide block: bf16 rows, weights kept in 32 bits, an odd row count
        dict(name="norm_train_97k_x1024_bf16", op="norm_train", rows=97001, channels=1024, dtype=BF16, params=F32),
        # rotation of one small set's heads: latency
        dict(name="rotary_450x4x64_f32", op="rotary", rows=450, heads=4, dim=64, dtype=F32, res=16,
             split=False, packed=False, inverse=False),
        # queries and keys rotated together inside a packed [rows, 3, heads, dim] projection, 63 of 64 pairs in use
        dict(name="rotary_packed_20k_x24x128_bf16", op="rotary", rows=20384, heads=24, dim=128, dtype=BF16, res=64,
             split=False, packed=True, inverse=False),
        # gradient of a large set's rotation, paired halves
        dict(name="rotary_inverse_400k_x24x128_bf16", op="rotary", rows=400311, heads=24, dim=128, dtype=BF16, res=256,
             split=True, packed=False, inverse=True),
        # attention of the smallest voxel set: latency
        dict(name="attention_450x4x32_f32", op="attention", queries=450, keys=0, entries=1, heads=4, kv_heads=4,
             dim=32, dtype=F32, empty=False),
        # self-attention inside many ragged windows of a 64^3 set
        dict(name="attention_windows_20k_x12x64_bf16", op="attention", queries=20384, keys=0, entries=161, heads=12,
             kv_heads=12, dim=64, dtype=BF16, empty=False),
        # full self-attention over one 64^3 structure (4.94 % occupancy)
        dict(name="attention_full_13k_x12x128_bf16", op="attention", queries=12948, keys=0, entries=1, heads=12,
             kv_heads=12, dim=128, dtype=BF16, empty=False),
        # a single query token per entry over all voxels of four 256^3 sets, shared key heads
        dict(name="attention_1q_1187k_x8x64_bf16", op="attention", queries=4, keys=1187403, entries=4, heads=8,
             kv_heads=2, dim=64, dtype=BF16, empty=False),
        # training step of self-attention, two ragged entries
        dict(name="attention_train_13k_x8x128_bf16", op="attention_train", queries=12948, keys=0, entries=2, heads=8,
             kv_heads=8, dim=128, dtype=BF16, empty=False),
        # training step of attention to a few conditioning tokens, one entry without any; 32-bit
        dict(name="attention_train_cross_20k_x4x64_f32", op="attention_train", queries=20384, keys=4111, entries=4,
             heads=4, kv_heads=4, dim=64, dtype=F32, empty=True),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "rotary", "attention", "attention_train"])
    dtype = rng.choice([F32, BF16])
    if op.startswith("norm"):
        channels = _log_int(rng, 8, 2560)
        if rng.random() < 0.6:
            channels = max(8, channels // 8 * 8)
        rows = max(2, _log_int(rng, 4000, 150_000_000) // channels)
        return dict(op=op, rows=rows, channels=channels, dtype=dtype, params=rng.choice([F32, dtype]))
    if op == "rotary":
        dim = rng.choice([16, 32, 48, 64, 80, 96, 128, 128, 2 * rng.randint(4, 64)])
        heads = _log_int(rng, 1, 32)
        rows = max(2, _log_int(rng, 4000, 300_000_000) // (heads * dim))
        return dict(op=op, rows=rows, heads=heads, dim=dim, dtype=dtype, res=rng.choice([16, 64, 128, 512]),
                    split=rng.random() < 0.5, packed=rng.random() < 0.3, inverse=rng.random() < 0.4)
    dim = rng.choice([32, 64, 64, 96, 128, 128, 8 * rng.randint(1, 16)])
    kv_heads = _log_int(rng, 1, 8)
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    entries = _log_int(rng, 1, 64)
    queries, keys = _log_int(rng, 1, 8192), _log_int(rng, 8, 65536)
    if rng.random() < 0.5:
        queries, keys = max(8, min(queries, 8192)), 0
    empty = keys > 0 and entries > 1 and rng.random() < 0.5
    while True:
        case = dict(op=op, queries=queries * entries, keys=keys * entries, entries=entries, heads=heads,
                    kv_heads=kv_heads, dim=dim, dtype=dtype, empty=empty)
        lq, lk = _lengths(case)
        if entries * heads * max(lq) * max(lk) <= 400_000_000:
            return case
        if queries > max(1, keys) and queries > 8:
            queries = max(8, queries // 2)
        elif keys > 8:
            keys = max(8, keys // 2)
        elif entries > 2:
            entries //= 2
        else:
            queries = max(8, queries // 2)


def _split(total, entries, seed):
    """Ragged lengths of `entries` parts with the sum `total`, the same for the same arguments."""
    rng = random.Random(seed)
    weights = [0.15 + rng.random() ** 2 for _ in range(entries)]
    ends, run_, whole = [], 0.0, sum(weights)
    for w in weights:
        run_ += w
        ends.append(int(total * run_ / whole + 0.5))
    ends[-1] = total
    return [e - b for b, e in zip([0] + ends[:-1], ends)]


def _lengths(case):
    """Queries and keys of each entry (keys = 0 in the case: self-attention)."""
    lq = _split(case["queries"], case["entries"], 1000003 * case["queries"] + case["entries"])
    if case["queries"] <= case["entries"]:
        lq = [1] * case["queries"] + [0] * (case["entries"] - case["queries"])
    if not case["keys"]:
        return lq, list(lq)
    parts = case["entries"] - (1 if case["empty"] else 0)
    lk = _split(case["keys"], parts, 7919 * case["keys"] + case["entries"])
    if case["empty"]:
        lk.insert(case["entries"] // 2, 0)  # the queries of this entry see no key at all
    return lq, lk


def _offsets(lengths):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    return ends


def _sections(dim):
    """Pairs for each of the three axes: equal parts, what is left over stays unrotated (63 of 64 at dim 128)."""
    return (dim // 2 // 3,) * 3


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, to=None):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(kind if to is None else to)

    if case["op"].startswith("norm"):
        n, c = case["rows"], case["channels"]
        p = _TYPES[case["params"]]
        # channels of unequal size and offset, as a residual stream has them
        spread = torch.exp(0.5 * torch.randn(c, generator=g, device="cuda"))
        x = torch.randn((n, c), generator=g, device="cuda").mul_(spread).add_(0.3 * spread)
        state = dict(op=case["op"], x=x.to(kind), weight=normal(c, std=0.2, mean=1.0, to=p), bias=normal(c, std=0.2, to=p), eps=1e-6)
        if case["op"] == "norm_train":
            state["grad"] = normal(n, c)
        return state
    if case["op"] == "rotary":
        n, h, d = case["rows"], case["heads"], case["dim"]
        coords = torch.randint(0, case["res"], (n, 4), generator=g, device="cuda", dtype=torch.int32)
        coords[:, 0] = 0
        sections = _sections(d)
        ladder = torch.arange(sections[0], device="cuda", dtype=torch.float64) / max(1, sections[0])
        freqs = (10000.0 ** -ladder).repeat(3).float()
        # packed: queries and keys are the first two thirds of one projection's rows
        x = normal(n, h // 2 * 3 if case["packed"] and h > 1 else h, d)
        if case["packed"] and h > 1:
            x = x[:, :h // 2 * 2]
        return dict(op="rotary", x=x, positions=coords[:, 1:], freqs=freqs, sections=sections, split=case["split"],
                    inverse=case["inverse"])
    lq, lk = _lengths(case)
    d = case["dim"]
    state = dict(op=case["op"], q=normal(sum(lq), case["heads"], d, std=1.3), k=normal(sum(lk), case["kv_heads"], d, std=1.3),
                 v=normal(sum(lk), case["kv_heads"], d), scale=d ** -0.5, most_queries=max(lq), most_keys=max(lk),
                 q_offsets=torch.tensor(_offsets(lq), dtype=torch.int32, device="cuda"),
                 k_offsets=torch.tensor(_offsets(lk), dtype=torch.int32, device="cuda"))
    if case["op"] == "attention_train":
        state["grad"] = normal(sum(lq), case["heads"], d)
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import submanifold_sparse_convolution_submconv3d_amd as sc
    if s["op"] == "norm":
        return sc.submconv_layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"])
    if s["op"] == "norm_train":
        y, stats = sc.submconv_layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], return_stats=True)
        dx, dw, db = sc.submconv_layer_norm_backward(s["grad"], s["x"], stats, s["weight"])
        return y, dx, dw, db
    if s["op"] == "rotary":
        return sc.submconv_rotary(s["x"], s["positions"], s["freqs"], s["sections"], split=s["split"], inverse=s["inverse"])
    if s["op"] == "attention":
        return sc.submconv_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], scale=s["scale"])
    out, lse = sc.submconv_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], scale=s["scale"], return_lse=True)
    dq, dk, dv = sc.submconv_attention_backward(s["grad"], s["q"], s["k"], s["v"], out, lse, s["q_offsets"], s["k_offsets"],
                                                scale=s["scale"])
    return out, dq, dk, dv


def _run_plain(s):
    if s["op"].startswith("norm"):
        return _plain_norm(s)
    if s["op"] == "rotary":
        return _plain_rotary(s)
    return _plain_attention(s)


def _plain_norm(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    kind, param = s["x"].dtype, s["weight"].dtype
    centred = x - x.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((centred * centred).mean(dim=1, keepdim=True) + s["eps"])
    hat = centred * rstd
    y = (hat * w + b).to(kind)
    if s["op"] == "norm":
        return y
    g = s["grad"].float()
    gw = g * w
    dx = rstd * (gw - gw.mean(dim=1, keepdim=True) - hat * (gw * hat).mean(dim=1, keepdim=True))
    return y, dx.to(kind), (g * hat).sum(dim=0).to(param), g.sum(dim=0).to(param)


def _plain_rotary(s):
    x, kind = s["x"].float(), s["x"].dtype
    d = x.shape[-1]
    n = sum(s["sections"])
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=x.device),
                                   torch.tensor(s["sections"], device=x.device), output_size=n)
    angle = s["positions"].float()[:, axis] * s["freqs"]
    if s["inverse"]:
        angle = -angle
    c, t = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :]
    if s["split"]:
        a, b = x[..., :n], x[..., d // 2:d // 2 + n]
        out = torch.cat([a * c - b * t, x[..., n:d // 2], a * t + b * c, x[..., d // 2 + n:]], dim=-1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        out = torch.cat([torch.stack([a * c - b * t, a * t + b * c], dim=-1).flatten(-2), x[..., 2 * n:]], dim=-1)
    return out.to(kind)


def _rows_of(offsets, most):
    """Row numbers [entries, most] of a ragged batch and which of them exist."""
    rows = offsets[:-1, None].long() + torch.arange(most, device=offsets.device)
    return rows, rows < offsets[1:, None]


def _plain_attention(s):
    kind = s["q"].dtype
    h, hk, d = s["q"].shape[1], s["k"].shape[1], s["q"].shape[2]
    group, entries = h // hk, s["q_offsets"].shape[0] - 1
    lq, lk = s["most_queries"], s["most_keys"]
    q_rows, q_there = _rows_of(s["q_offsets"], lq)
    k_rows, k_there = _rows_of(s["k_offsets"], lk)

    def pad_q(t):  # [entries, kv heads, group * queries, dim]
        t = t.float()[q_rows.clamp(max=t.shape[0] - 1)].mul_(q_there[..., None, None])
        return t.reshape(entries, lq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(entries, hk, group * lq, d)

    def pad_k(t):
        return t.float()[k_rows.clamp(max=t.shape[0] - 1)].mul_(k_there[..., None, None]).permute(0, 2, 1, 3)

    def unpad_q(t):
        return t.reshape(entries, hk, group, lq, d).permute(0, 3, 1, 2, 4).reshape(entries, lq, h, d)[q_there].to(kind)

    def unpad_k(t):
        return t.permute(0, 2, 1, 3)[k_there].to(kind)

    q, k, v = pad_q(s["q"]), pad_k(s["k"]), pad_k(s["v"])
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    p.masked_fill_(~k_there[:, None, None, :], -math.inf)
    p.sub_(p.amax(dim=3, keepdim=True).clamp_(min=-3e38)).exp_()
    total = p.sum(dim=3, keepdim=True)
    p.div_(total.clamp_(min=1e-38))  # a row without keys stays zero
    out = torch.matmul(p, v)
    if s["op"] == "attention":
        return unpad_q(out)
    g = pad_q(s["grad"])
    dv = torch.matmul(p.transpose(2, 3), g)
    ds = torch.matmul(g, v.transpose(2, 3).contiguous()).sub_((g * out).sum(dim=3, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    return unpad_q(out), unpad_q(dq), unpad_k(dk), unpad_k(dv)


def work(case):
    size = 4 if case["dtype"] == F32 else 2
    if case["op"].startswith("norm"):
        n, c = case["rows"], case["channels"]
        train = case["op"] == "norm_train"
        return {"bytes": n * c * size * (4 if train else 2) + 4 * c * (4 if train else 2), "flops": n * c * (20 if train else 8)}
    if case["op"] == "rotary":
        h = case["heads"] // 2 * 2 if case["packed"] and case["heads"] > 1 else case["heads"]
        e = case["rows"] * h * case["dim"]
        return {"bytes": 2 * e * size + 12 * case["rows"], "flops": 3 * e}
    lq, lk = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    products = sum(a * b for a, b in zip(lq, lk)) * h * d * 2
    if case["op"] == "attention":
        return {"bytes": size * d * (2 * sum(lq) * h + 2 * sum(lk) * hk), "flops": 2 * products}
    return {"bytes": size * d * (4 * sum(lq) * h + 4 * sum(lk) * hk), "flops": 7 * products}


# ----------------------------------------------------------------------------
# 64 bits, from the definitions
# ----------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    return _exact_attention(case, s)


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    sigma = torch.sqrt(var + s["eps"])
    x = (x - mean) / sigma
    y = torch.addcmul(s["bias"].double(), x, w)
    if s["op"] == "norm":
        return y
    g = s["grad"].double()
    # dL/dx = (I - 1 1^T / C - hat hat^T / C) (g w) / sigma
    along = torch.einsum("nc,nc,c->n", g, x, w)[:, None] / x.shape[1]
    mid = torch.mv(g, w)[:, None] / x.shape[1]
    return y, (g * w - mid - x * along) / sigma, torch.einsum("nc,nc->c", g, x), g.sum(0)


def _exact_rotary(s):
    x = s["x"].double()
    n, h, d = x.shape
    pairs = x.reshape(n, h, 2, d // 2).transpose(2, 3) if s["split"] else x.reshape(n, h, d // 2, 2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = torch.zeros((n, d // 2), dtype=torch.float64, device=x.device)
    first = 0
    for axis, count in enumerate(s["sections"]):
        angle[:, first:first + count] = s["positions"][:, axis, None].double() * s["freqs"][first:first + count].double()
        first += count
    z = z * torch.polar(torch.ones_like(angle), -angle if s["inverse"] else angle)[:, None, :]
    out = torch.view_as_real(z)
    return (out.transpose(2, 3) if s["split"] else out).reshape(n, h, d)


def _exact_attention(case, s):
    lq, lk = _lengths(case)
    train = case["op"] == "attention_train"
    group = case["heads"] // case["kv_heads"]
    q, k, v = (s[n].double().transpose(0, 1).contiguous() for n in ("q", "k", "v"))
    out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    g = s["grad"].double().transpose(0, 1).contiguous() if train else None
    q0 = k0 = 0
    for nq, nk in zip(lq, lk):
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        if not nq or not nk:
            continue
        # a few heads at a time, so that the score matrices stay small
        step = max(1, 400_000_000 // (nq * nk * group))
        for h0 in range(0, case["kv_heads"], step):
            ks = slice(h0, min(case["kv_heads"], h0 + step))
            many = ks.stop - ks.start
            qs = slice(ks.start * group, ks.stop * group)
            qq = q[qs, a].reshape(many, group * nq, -1)
            p = torch.softmax(torch.baddbmm(qq.new_zeros(()), qq, k[ks, b].mT.contiguous(), beta=0, alpha=s["scale"]), dim=2)
            o = torch.bmm(p, v[ks, b])
            out[qs, a] = o.reshape(many * group, nq, -1)
            if train:
                gg = g[qs, a].reshape(many, group * nq, -1)
                dp = torch.bmm(gg, v[ks, b].mT.contiguous())
                ds = p * (dp - (dp * p).sum(2, keepdim=True)) * s["scale"]
                dq[qs, a] = torch.bmm(ds, k[ks, b]).reshape(many * group, nq, -1)
                dk[ks, b] = torch.bmm(ds.mT.contiguous(), qq)
                dv[ks, b] = torch.bmm(p.mT.contiguous(), gg)
    if not train:
        return out.transpose(0, 1)
    return tuple(t.transpose(0, 1) for t in (out, dq, dk, dv))
