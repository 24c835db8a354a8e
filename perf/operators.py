"""Workloads of the operators around the attention calls: the per-head norm with the position rotation (forward and
gradient), the append of new tokens to a paged cache (16-bit and 8-bit pages), and decode attention over 8-bit pages.

``run`` computes a case in its plain form, elementary torch operations in 32 bits, or with ``own`` by the package's calls.
"""
import math
import random

import torch

own = False

BLOCK = 64
EPS = 1e-6
THETA = 1e6
E4M3_MAX = 448.0
MIN_EXP = -64          # 8-bit pages: no scale under 2^-64
HEADS = ((32, 8, 128), (40, 8, 128), (8, 2, 128), (8, 1, 128), (4, 4, 128), (2, 1, 64))
DECODE_HEADS = ((32, 8), (40, 8), (8, 2), (8, 1), (4, 4), (8, 8))


def listed():
    return [
        # one small layer in fp32, where the launch is what counts
        dict(name="norm-rope fwd tiny f32", op="norm_rope", dir="fwd", dtype="f32", seqs=1, tokens=512, packed=False,
             hq=2, hkv=1, d=64),
        # the query/key preparation of one 8k training sequence, read out of the fused projection
        dict(name="norm-rope fwd 8k", op="norm_rope", dir="fwd", dtype="bf16", seqs=1, tokens=8192, packed=False,
             hq=32, hkv=8, d=128),
        # its gradient for two 32k sequences of a 40-head layer
        dict(name="norm-rope bwd 2x32k", op="norm_rope", dir="bwd", dtype="bf16", seqs=2, tokens=32768, packed=False,
             hq=40, hkv=8, d=128),
        # the gradient for a packed batch of odd lengths in fp32
        dict(name="norm-rope bwd packed f32", op="norm_rope", dir="bwd", dtype="f32", seqs=5, tokens=611, packed=True,
             hq=8, hkv=2, d=64),
        # one new token of one sequence
        dict(name="append 1 token", op="append", bits=16, seqs=1, new_min=1, new_max=1, start_max=8191, hq=32, hkv=8,
             d=128, pool=True),
        # one step of 64 sequences into 8-bit pages
        dict(name="append 64 tokens q8", op="append", bits=8, seqs=64, new_min=1, new_max=1, start_max=65535, hq=32,
             hkv=8, d=128, pool=True),
        # a whole 8k prompt
        dict(name="append 8k prompt", op="append", bits=16, seqs=1, new_min=8192, new_max=8192, start_max=0, hq=32,
             hkv=8, d=128, pool=False),
        # pieces of prompts of any length behind what is cached, 8-bit pages
        dict(name="append ragged q8", op="append", bits=8, seqs=7, new_min=1, new_max=5000, start_max=999, hq=40,
             hkv=8, d=128, pool=False),
        # one sequence at 8k, K = 16
        dict(name="decode q8 1x8k", op="decode", seqs=1, min_hist=128, max_hist=128, k=16, hq=32, hkv=8),
        # 64 sequences at 8k to 64k, K = 32
        dict(name="decode q8 64 seqs", op="decode", seqs=64, min_hist=128, max_hist=1024, k=32, hq=32, hkv=8),
        # short and empty histories, five query heads for each KV head
        dict(name="decode q8 ragged", op="decode", seqs=5, min_hist=0, max_hist=40, k=8, hq=40, hkv=8),
        # every block of eight 64k sequences
        dict(name="decode q8 all history", op="decode", seqs=8, min_hist=1024, max_hist=1024, k=1024, hq=32, hkv=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "decode"))
    if op == "norm_rope":
        hq, hkv, d = rng.choice(HEADS)
        return dict(op=op, dir=rng.choice(("fwd", "bwd")), dtype=rng.choice(("bf16", "bf16", "f32")),
                    seqs=rng.randint(1, 4), tokens=_log_int(rng, 1, 8192), packed=rng.random() < 0.5,
                    hq=hq, hkv=hkv, d=d)
    if op == "append":
        hq, hkv, d = rng.choice(HEADS)
        bits = rng.choice((8, 16))
        if rng.random() < 0.5:
            return dict(op=op, bits=bits, seqs=_log_int(rng, 1, 256), new_min=1, new_max=1,
                        start_max=rng.choice((100, 8191, 65535)), hq=hq, hkv=hkv, d=d, pool=True)
        seqs = rng.randint(1, 6)
        top = _log_int(rng, 2, 6000)
        return dict(op=op, bits=bits, seqs=seqs, new_min=1, new_max=top, start_max=rng.choice((0, 63, 4000)),
                    hq=hq, hkv=hkv, d=d, pool=False)
    hq, hkv = rng.choice(DECODE_HEADS)
    seqs = _log_int(rng, 1, 64)
    top = _log_int(rng, 1, min(1024, 24576 // seqs))
    return dict(op=op, seqs=seqs, min_hist=rng.randint(0, top), max_hist=top, k=rng.randint(0, 64), hq=hq, hkv=hkv)


# ------------------------------------------------------------------------------------------------------- sizes
def _lengths(case):
    """Lengths of a case, the same for every seed of its values."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["seqs"]
    if case["op"] == "norm_rope":
        if not case["packed"]:
            return [case["tokens"]] * n
        return [r.randint(max(1, case["tokens"] // 2), case["tokens"]) for _ in range(n)]
    if case["op"] == "append":
        new = [_log_int(r, case["new_min"], case["new_max"]) if case["new_max"] > case["new_min"] else case["new_max"]
               for _ in range(n)]
        return new, [r.randint(0, case["start_max"]) for _ in range(n)]
    return [r.randint(case["min_hist"], case["max_hist"]) * BLOCK + r.randint(1, BLOCK) for _ in range(n)]


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        lens, d = _lengths(case), case["d"]
        t, pos = sum(lens), max(lens)
        n = t * (hq + hkv) * d
        if case["dir"] == "fwd":
            return dict(bytes=2 * n * e + pos * d * 4 + 2 * d * e, flops=8 * n)
        return dict(bytes=3 * n * e + pos * d * 4 + 2 * d * e + 2 * d * 4, flops=16 * n)
    if case["op"] == "append":
        (new, start), d = _lengths(case), case["d"]
        t = sum(new)
        pos = len({p for n, s in zip(new, start) for p in range(s, s + n)})
        by = t * (2 * hq + 2 * hkv) * d * 2 + 2 * t * hkv * d * (case["bits"] // 8) + pos * d * 4
        if case["pool"]:                                  # filled pages: their older rows, and the mean
            fills = sum((s + n) // BLOCK - s // BLOCK for n, s in zip(new, start))
            by += fills * hkv * d * (BLOCK * (case["bits"] // 8) + 4)
        return dict(bytes=by, flops=8 * t * (hq + 2 * hkv) * d)
    kept = sum(min(case["k"], (n - 1) // BLOCK) * BLOCK + (n - 1) % BLOCK + 1 for n in _lengths(case))
    rows = case["seqs"] * hq * 128
    return dict(bytes=kept * hkv * 2 * 128 + rows * 4, flops=4 * kept * hq * 128)


# ------------------------------------------------------------------------------------------------------- inputs
def _table(rows, d):
    """cos and sin of each position's angles, [rows, d] fp32 (cos first), from 64-bit angles."""
    inv = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), dim=1).float()


def _cu(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def _projection(g, t, hq, hkv, d, dtype):
    """The fused projection's output and its q, k, v parts (strided by token)."""
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda", dtype=dtype)
    q, k, v = qkv.split((hq * d, hkv * d, hkv * d), dim=1)
    return q.view(t, hq, d), k.view(t, hkv, d), v.view(t, hkv, d)


def _weights(g, d, dtype):
    return [(1 + 0.25 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]


def _codes(g, shape):
    """8-bit pages as an append leaves them: values up to 448, a power of two for each page and head."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for i in range(0, shape[0], 4096):
        x = torch.randn((min(4096, shape[0] - i),) + shape[1:], generator=g, device="cuda", dtype=torch.bfloat16)
        out[i:i + 4096] = x.mul_(80).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    scale = torch.randint(-9, -4, shape[:2], generator=g, device="cuda").float().exp2()
    return out, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "norm_rope":
        d, lens = case["d"], _lengths(case)
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        t = sum(lens)
        q, k, _ = _projection(g, t, hq, hkv, d, dt)
        st = dict(case=case, table=_table(max(lens), d), w=_weights(g, d, dt), pos=None)
        if case["packed"]:
            st["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
        else:
            q, k = q.view(case["seqs"], -1, hq, d), k.view(case["seqs"], -1, hkv, d)
        st.update(q=q, k=k)
        if case["dir"] == "bwd":
            st["dq"] = torch.randn(q.shape, generator=g, device="cuda", dtype=dt)
            st["dk"] = torch.randn(k.shape, generator=g, device="cuda", dtype=dt)
        return st
    if case["op"] == "append":
        d = case["d"]
        new, start = _lengths(case)
        n, t = len(new), sum(new)
        q, k, v = _projection(g, t, hq, hkv, d, torch.bfloat16)
        first = [s // BLOCK for s in start]
        last = [(s + m - 1) // BLOCK for s, m in zip(start, new)]
        own_pages = sum(b - a + 1 for a, b in zip(first, last))
        perm = (torch.randperm(own_pages, generator=torch.Generator().manual_seed(seed)) + 1).tolist()
        ptab = [[0] * (max(last) + 1) for _ in range(n)]         # older blocks: page 0, which no call touches
        for i in range(n):
            for b in range(first[i], last[i] + 1):
                ptab[i][b] = perm.pop()
        shape = (own_pages + 1, hkv, BLOCK, d)
        st = dict(case=case, q=q, k=k, v=v, table=_table(max(s + m for s, m in zip(start, new)), d),
                  w=_weights(g, d, torch.bfloat16), page_table=torch.tensor(ptab, dtype=torch.int32).cuda(),
                  kv_len=torch.tensor([s + m for s, m in zip(start, new)], dtype=torch.int32).cuda(),
                  cu=None if case["new_max"] == 1 else _cu(new), max_new=max(new),
                  kpool=torch.zeros((shape[0], hkv, d), device="cuda") if case["pool"] else None)
        if case["bits"] == 8:
            (st["kc"], st["ks"]), (st["vc"], st["vs"]) = _codes(g, shape), _codes(g, shape)
        else:
            st["kc"], st["vc"] = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
                                  for _ in range(2))
        return st
    lens, n, K = _lengths(case), case["seqs"], case["k"]
    pages = [(m + BLOCK - 1) // BLOCK for m in lens]
    perm = torch.randperm(sum(pages), generator=g, device="cuda").to(torch.int32)
    ptab = torch.zeros((n, max(pages)), dtype=torch.int32, device="cuda")
    for i, m in enumerate(pages):
        ptab[i, :m] = perm[sum(pages[:i]):sum(pages[:i]) + m]
    kc, ks = _codes(g, (sum(pages), hkv, BLOCK, 128))
    vc, vs = _codes(g, (sum(pages), hkv, BLOCK, 128))
    kv_len = torch.tensor(lens, dtype=torch.int32).cuda()
    nh = ((kv_len - 1) // BLOCK)[:, None]
    s = torch.randn((n, hkv, max(pages)), generator=g, device="cuda")
    s = s.masked_fill(torch.arange(max(pages), device="cuda") >= nh[:, :, None], -math.inf)
    kk = min(K, max(pages))
    val, idx = s.topk(kk, dim=2)
    idx = idx.masked_fill(val == -math.inf, 1 << 30).sort(dim=2).values
    gate = torch.gather(s, 2, idx.clamp(max=max(pages) - 1)) - s.double().logsumexp(2, keepdim=True).float()
    gate = gate.masked_fill(idx == 1 << 30, -math.inf)
    idx = idx.masked_fill(idx == 1 << 30, -1).to(torch.int32)
    pad = (0, K - kk)
    return dict(case=case, q=torch.randn((n, hq, 128), generator=g, device="cuda", dtype=torch.bfloat16), kc=kc, ks=ks,
                vc=vc, vs=vs, page_table=ptab, kv_len=kv_len,
                idx=torch.nn.functional.pad(idx, pad, value=-1).contiguous(),
                cnt=nh.clamp(max=K).expand(n, hkv).to(torch.int32).contiguous(),
                gate=torch.nn.functional.pad(gate, pad, value=-math.inf).contiguous())


# ------------------------------------------------------------------------------------------------------- plain forms
def _rows(table, pos):
    c, s = table[pos.long()].chunk(2, dim=-1)
    return c.unsqueeze(-2), s.unsqueeze(-2)


def _positions(st):
    if st["pos"] is not None:
        return st["pos"]
    return torch.arange(st["q"].shape[1], device="cuda").expand(st["q"].shape[0], -1)


def _norm_rope(x, w, cos, sin):
    x = x.float()
    a, b = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()).chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _norm_rope_grad(x, dy, w, cos, sin):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    a, b = dy.float().chunk(2, dim=-1)
    gn = torch.cat((a * cos + b * sin, b * cos - a * sin), dim=-1)
    g = gn * w.float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (gn * xh).flatten(0, -2).sum(0)


def _plain_norm_rope(st):
    cos, sin = _rows(st["table"], _positions(st))
    dt = st["q"].dtype
    if st["case"]["dir"] == "fwd":
        return dict(q=_norm_rope(st["q"], st["w"][0], cos, sin).to(dt), k=_norm_rope(st["k"], st["w"][1], cos, sin).to(dt))
    dq, dwq = _norm_rope_grad(st["q"], st["dq"], st["w"][0], cos, sin)
    dk, dwk = _norm_rope_grad(st["k"], st["dk"], st["w"][1], cos, sin)
    return dict(dq=dq.to(dt), dk=dk.to(dt), dq_weight=dwq, dk_weight=dwk)


def _places(st):
    """For each new token its position; for each page row the token that is written there (or -1)."""
    t = st["q"].shape[0]
    tok = torch.arange(t, device="cuda")
    if st["cu"] is None:
        seq, pos = tok, st["kv_len"].long() - 1
    else:
        cu = st["cu"].long()
        seq = torch.bucketize(tok, cu[1:], right=True)
        pos = tok - cu[seq + 1] + st["kv_len"].long()[seq]
    page = st["page_table"][seq, pos // BLOCK].long()
    row = torch.full((st["kc"].shape[0] * BLOCK,), -1, device="cuda", dtype=torch.long)
    row[page * BLOCK + pos % BLOCK] = tok
    return pos, row.view(-1, BLOCK)


def _store(cache, scale, new, row):
    """New rows into 8-bit pages: the scale grows where they need it, older rows are expressed in it."""
    has = row >= 0
    first = torch.where(has, torch.arange(BLOCK, device="cuda"), BLOCK).amin(1)
    old = (torch.arange(BLOCK, device="cuda") < first[:, None]) & has.any(1, keepdim=True)
    val = torch.where(has[:, :, None, None], new[row.clamp(min=0)], 0.0).transpose(1, 2)
    amax = val.abs().amax((2, 3))
    m, e = torch.frexp(amax)
    need = torch.ldexp(torch.ones_like(amax), (e - torch.where(m <= 0.875, 9, 8)).clamp(min=MIN_EXP))
    need = torch.where(amax > 0, need, 2.0 ** MIN_EXP)
    keep = (first[:, None] > 0) & (amax <= E4M3_MAX * scale)
    s = torch.where(keep, scale, need)
    s = torch.where(has.any(1, keepdim=True), s, scale)
    codes = torch.where(has[:, None, :, None], val / s[:, :, None, None],
                        cache.float() * (scale / s)[:, :, None, None]).to(torch.float8_e4m3fn)
    cache.view(torch.uint8).copy_(torch.where((has | old)[:, None, :, None], codes.view(torch.uint8),
                                              cache.view(torch.uint8)))
    scale.copy_(s)


def _plain_append(st):
    pos, row = _places(st)
    cos, sin = _rows(st["table"], pos)
    qo = _norm_rope(st["q"], st["w"][0], cos, sin).to(torch.bfloat16)
    k = _norm_rope(st["k"], st["w"][1], cos, sin)
    v = st["v"].float()
    out = dict(q=qo, k_cache=st["kc"], v_cache=st["vc"])
    if st["case"]["bits"] == 8:
        _store(st["kc"], st["ks"], k, row)
        _store(st["vc"], st["vs"], v, row)
        out.update(k_scale=st["ks"], v_scale=st["vs"])
    else:
        has = (row >= 0)[:, None, :, None]
        at = row.clamp(min=0)
        st["kc"].copy_(torch.where(has, k.to(torch.bfloat16)[at].transpose(1, 2), st["kc"]))
        st["vc"].copy_(torch.where(has, st["v"][at].transpose(1, 2), st["vc"]))
    if st["kpool"] is not None:
        mean = st["kc"].float().mean(2)
        if st["case"]["bits"] == 8:
            mean = mean * st["ks"][:, :, None]
        st["kpool"].copy_(torch.where((row[:, -1] >= 0)[:, None, None], mean, st["kpool"]))
        out["kpool"] = st["kpool"]
    return out


def _kept(st):
    """The kept blocks of each (sequence, KV head), the current one last: page, gate, tokens."""
    n, h, K = st["idx"].shape
    kv = st["kv_len"].long()
    cur = ((kv - 1) // BLOCK)[:, None, None].expand(n, h, 1)
    blk = torch.cat((st["idx"].long().clamp(min=0), cur), dim=2)
    page = torch.gather(st["page_table"].long()[:, None].expand(n, h, -1), 2, blk)
    gate = torch.cat((st["gate"], torch.zeros((n, h, 1), device="cuda")), dim=2)
    used = torch.arange(K, device="cuda") < st["cnt"][:, :, None]
    size = torch.where(used, BLOCK, 0)
    size = torch.cat((size, (kv[:, None, None] - cur * BLOCK)), dim=2)
    return page, gate, size


def _plain_decode(st):
    page, gate, size = _kept(st)
    n, h, kb = page.shape
    d = st["q"].shape[-1]
    head = torch.arange(h, device="cuda")[None, :, None]
    q = st["q"].float().view(n, h, -1, d)
    k = (st["kc"][page, head].float() * st["ks"][page, head][..., None, None]).view(n, h, kb * BLOCK, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(n, h, -1, kb, BLOCK) / math.sqrt(d)
    live = torch.arange(BLOCK, device="cuda") < size[..., None]
    x = torch.where(live[:, :, None], x + gate[:, :, None, :, None], -math.inf).flatten(3)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = (st["vc"][page, head].float() * st["vs"][page, head][..., None, None]).view(n, h, kb * BLOCK, d)
    o = torch.matmul(p / l, v).view(n, -1, d).to(torch.bfloat16)
    return dict(o=o, lse=(m + torch.log(l)).view(n, -1))


def _own(st):
    from trainable_gated_block_b200 import sas
    op = st["case"]["op"]
    if op == "norm_rope":
        if st["case"]["dir"] == "fwd":
            q, k = sas.qk_norm_rope(st["q"], st["k"], st["table"], st["w"][0], st["w"][1], positions=st["pos"], eps=EPS)
            return dict(q=q, k=k)
        dq, dk, dwq, dwk = sas.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["table"], st["w"][0],
                                                st["w"][1], positions=st["pos"], eps=EPS)
        return dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk)
    if op == "append":
        out = dict(k_cache=st["kc"], v_cache=st["vc"])
        more = dict(q_weight=st["w"][0], k_weight=st["w"][1], cu_new=st["cu"], max_new=st["max_new"], eps=EPS,
                    kpool=st["kpool"])
        if st["case"]["bits"] == 8:
            out["q"] = sas.append_paged_q8(st["q"], st["k"], st["v"], st["table"], st["kc"], st["vc"], st["ks"],
                                           st["vs"], st["page_table"], st["kv_len"], **more)
            out.update(k_scale=st["ks"], v_scale=st["vs"])
        else:
            out["q"] = sas.append_paged(st["q"], st["k"], st["v"], st["table"], st["kc"], st["vc"], st["page_table"],
                                        st["kv_len"], **more)
        if st["kpool"] is not None:
            out["kpool"] = st["kpool"]
        return out
    o, lse = sas.decode_paged_q8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["page_table"], st["kv_len"],
                                 st["idx"], st["cnt"], st["gate"])
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _own(state)
    return dict(norm_rope=_plain_norm_rope, append=_plain_append, decode=_plain_decode)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------- in 64 bits
def _turn(x, angle_row, back=False):
    """Complex numbers (x_i, x_{i + d/2}) times e^{i angle} (or its conjugate)."""
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half], x[..., half:])
    w = torch.complex(angle_row[..., :half].double(), angle_row[..., half:].double())
    z = z * (w.conj() if back else w)
    return torch.cat((z.real, z.imag), dim=-1)


def _exact_rows(x, w, angle):
    x = x.double()
    inv = 1 / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    return _turn(x * inv * w.double(), angle[..., None, :])


def _exact_rows_grad(x, dy, w, angle):
    """The norm's Jacobian w_i (delta_ij r - x_i x_j r^3 / d), transposed, behind the rotation's transpose."""
    x, gn = x.double(), _turn(dy.double(), angle[..., None, :], back=True)
    r = 1 / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    wg = gn * w.double()
    dx = wg * r - x * (wg * x).sum(-1, keepdim=True) * r.pow(3) / x.shape[-1]
    return dx, torch.einsum("rd,rd->d", gn.reshape(-1, x.shape[-1]), (x * r).reshape(-1, x.shape[-1]))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        n, s = (1, st["q"].shape[0]) if case["packed"] else st["q"].shape[:2]
        angle = st["table"][st["pos"].long()] if case["packed"] else st["table"][None, :s].expand(n, s, -1)
        if case["dir"] == "fwd":
            return dict(q=_exact_rows(st["q"], st["w"][0], angle), k=_exact_rows(st["k"], st["w"][1], angle))
        dq, dwq = _exact_rows_grad(st["q"], st["dq"], st["w"][0], angle)
        dk, dwk = _exact_rows_grad(st["k"], st["dk"], st["w"][1], angle)
        return dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk)
    if case["op"] == "append":
        return _exact_append(case, st)
    return _exact_decode(case, st)


def _exact_append(case, st):
    """Page by page: the values before their last rounding (the pooled mean: of the rounded ones)."""
    new, start = _lengths(case)
    pos = torch.cat([torch.arange(s, s + n) for n, s in zip(new, start)]).cuda()
    angle = st["table"][pos]
    k = _exact_rows(st["k"], st["w"][1], angle)
    out = dict(q=_exact_rows(st["q"], st["w"][0], angle))
    ptab = st["page_table"].tolist()
    pools = None if st["kpool"] is None else st["kpool"].double()
    for name, x, cache in (("k", k, st["kc"]), ("v", st["v"].double(), st["vc"])):
        whole = cache.double()
        scale = st[name + "s"].double() if case["bits"] == 8 else None
        tok = 0
        for i in range(len(new)):
            at, end = start[i], start[i] + new[i]
            while at < end:
                b = at // BLOCK
                upto, lo, p = min(end, (b + 1) * BLOCK), at % BLOCK, ptab[i][b]
                rows = x[tok:tok + upto - at].transpose(0, 1)            # [heads, rows, d]
                if case["bits"] == 8:
                    top = rows.abs().amax((1, 2))
                    need = torch.log2(top / E4M3_MAX).ceil().clamp(min=MIN_EXP).exp2()
                    s = torch.where(top <= scale[p] * E4M3_MAX, scale[p], need) if lo else need
                    whole[p, :, :lo] *= (scale[p] / s)[:, None, None]
                    whole[p, :, lo:lo + upto - at] = rows / s[:, None, None]
                    scale[p] = s
                else:
                    whole[p, :, lo:lo + upto - at] = rows
                if name == "k" and pools is not None and upto % BLOCK == 0:
                    kept = whole[p].float().to(cache.dtype).double().mean(1)
                    pools[p] = kept * scale[p][:, None] if case["bits"] == 8 else kept
                tok += upto - at
                at = upto
        out[name + "_cache"] = whole
        if scale is not None:
            out[name + "_scale"] = scale
    if pools is not None:
        out["kpool"] = pools
    return out


def _exact_decode(case, st):
    """One sequence at a time over the tokens that it keeps."""
    lens = _lengths(case)
    n, hq, d = st["q"].shape
    hkv = st["kc"].shape[1]
    o = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((n, hq), dtype=torch.float64, device="cuda")
    cnt = st["cnt"].tolist()
    for i in range(n):
        cur = (lens[i] - 1) // BLOCK
        q = st["q"][i].double().view(hkv, -1, d)
        for h in range(hkv):
            c = cnt[i][h]
            pages = torch.cat((st["page_table"][i][st["idx"][i, h, :c].long()], st["page_table"][i, cur:cur + 1])).long()
            tokens = c * BLOCK + lens[i] - cur * BLOCK
            keys = (st["kc"][pages, h].double() * st["ks"][pages, h, None, None].double()).view(-1, d)[:tokens]
            vals = (st["vc"][pages, h].double() * st["vs"][pages, h, None, None].double()).view(-1, d)[:tokens]
            bias = torch.zeros(tokens, dtype=torch.float64, device="cuda")
            bias[:c * BLOCK] = st["gate"][i, h, :c].double().repeat_interleave(BLOCK)
            x = q[h] @ keys.T / d ** 0.5 + bias
            z = x.logsumexp(1)
            g = q.shape[1]
            o[i, h * g:(h + 1) * g] = (x - z[:, None]).exp() @ vals
            lse[i, h * g:(h + 1) * g] = z
    return dict(o=o, lse=lse)
