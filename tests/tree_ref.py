"""Plain 64-bit forms of the tree operators, and inputs for their tests."""

import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make_case(past, n, H, Hk, D, bs, dtype=torch.float16, max_draft=None, window=-1, softcap=0.0, scale=0.0,
              slopes=False, sink=False, mask="tree", positions=True, pad=0, unmap=(), seed=0, q_std=1.5):
    """One step on the CPU.  Pool slots that hold no key are NaN.  mask: "tree" (random parents), "none" (NULL),
    "random" (any bits, some rows empty).  unmap: (b, page) entries set to -1.  pad: rows behind the last one."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(past), sum(n) + pad
    max_draft = max_draft or max(max(n), 1)
    words = -(-max_draft // 32)
    need = [-(-(p + m) // bs) for p, m in zip(past, n)]
    MB, NB = max(max(need), 1), sum(need) + 3
    perm = torch.randperm(NB, generator=g).int()
    table, at = torch.full((B, MB), -1, dtype=torch.int32), 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    pools = torch.full((2, NB * bs, Hk, D), float("nan"), dtype=dtype)
    for b in range(B):
        for p in range(past[b] + n[b]):
            pools[:, int(table[b, p // bs]) * bs + p % bs] = torch.randn(2, Hk, D, generator=g).to(dtype)
    for b, page in unmap:
        table[b, page] = -1
    cum = torch.zeros(B + 1, dtype=torch.int32)
    cum[1:] = torch.tensor(n).cumsum(0)
    pos, rows = torch.zeros(T, dtype=torch.int32), torch.zeros(T, max_draft, dtype=torch.bool)
    for b in range(B):
        depth = []
        for j in range(n[b]):
            t = int(cum[b]) + j
            if mask == "none":
                rows[t, :j + 1] = True
                depth.append(j)
                continue
            parent = int(torch.randint(max(0, j - 5), j, (1,), generator=g)) if j else -1
            depth.append(depth[parent] + 1 if j else 0)
            if j:
                rows[t] = rows[int(cum[b]) + parent]
            rows[t, j] = True
        if mask == "random":
            rows[int(cum[b]):int(cum[b]) + n[b]] = torch.rand(n[b], max_draft, generator=g) < 0.4
            if n[b]:
                rows[int(cum[b]) + n[b] // 2] = False
        for j, d in enumerate(depth):
            pos[int(cum[b]) + j] = past[b] + (d if positions else j)
    packed = torch.zeros(T, words, dtype=torch.int64)
    for i in range(max_draft):
        packed[:, i // 32] |= rows[:, i].long() << (i % 32)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    c = dict(past=past, n=n, H=H, Hk=Hk, D=D, bs=bs, NB=NB, MB=MB, B=B, T=T, max_draft=max_draft, window=window,
             softcap=softcap, scale=scale, dtype=dtype, rows=rows, cum=cum,
             past_t=torch.tensor(past, dtype=torch.int32), table=table, pos=pos,
             query=(q_std * torch.randn(T, H * D, generator=g)).to(dtype),
             key_cache=pools[0].view(NB, bs, Hk, D).clone(), value_cache=pools[1].view(NB, bs, Hk, D).clone(),
             mask=None if mask == "none" else packed, positions=pos if positions else None,
             slopes=(0.5 ** torch.arange(1, H + 1).float().clamp(max=8)) if slopes else None,
             sink=(2 * torch.randn(H, generator=g)).to(dtype) if sink else None)
    return c


def attention(c):
    """(output, tolerance), both [T, H, D] in 64 bits; NaN tolerance never occurs.  Rows of padding are None.

    Tolerance, with u the half step of the 16-bit type and A = sum p |v| (the output's own absolute sum):
      u A        P rounded to 16 bits for P V
      u |o|      the output's rounding
      2 w A      w: relative error of a weight.  A score is D products summed in fp32, an error of at most
                 (D + 8) 2^-24 sum |q k| scale (the 8: scaling, softcap's arithmetic on a result no larger, the
                 bias and the maximum's subtraction at |x| each), its exponential 2^-21 relative; numerator and
                 denominator each carry it
      fp16 only: P below 2^-14 is subnormal, off by 2^-25 for each key against a row sum >= 1: keys 2^-25 max|v|."""
    H, Hk, D, bs, dtype = c["H"], c["Hk"], c["D"], c["bs"], c["dtype"]
    u, G = HALF_STEP[dtype], c["H"] // c["Hk"]
    scale = c["scale"] or 1 / math.sqrt(D)
    out, tol = torch.zeros(c["T"], H, D).double(), torch.zeros(c["T"], H, D).double()
    q = c["query"].double().view(c["T"], H, D)
    K, V = (c[k].double().view(-1, Hk, D) for k in ("key_cache", "value_cache"))
    for b in range(c["B"]):
        past, n, t0 = c["past"][b], c["n"][b], int(c["cum"][b])
        keys = [p for p in range(past + n) if int(c["table"][b, p // bs]) >= 0]
        slots = torch.tensor([int(c["table"][b, p // bs]) * bs + p % bs for p in keys], dtype=torch.long)
        for j in range(n):
            t = t0 + j
            qpos = int(c["pos"][t]) if c["positions"] is not None else past + j
            see, kpos = [], []
            for p in keys:
                kp = p
                if p >= past:
                    kp = int(c["pos"][t0 + p - past]) if c["positions"] is not None else p
                ok = p < past or bool(c["rows"][t, p - past])
                if c["window"] > 0 and kp <= max(qpos, past) - c["window"]:
                    ok = False
                see.append(ok)
                kpos.append(kp)
            see = torch.tensor(see, dtype=torch.bool)
            if not see.any():
                continue
            kp = torch.tensor(kpos, dtype=torch.float64)[see]
            for h in range(H):
                k, v = K[slots[see], h // G], V[slots[see], h // G]
                x = (k @ q[t, h]) * scale
                size = (k.abs() @ q[t, h].abs()) * scale
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                    size = size + 2 * c["softcap"]
                if c["slopes"] is not None:
                    x = x + float(c["slopes"][h]) * (kp - qpos)
                    size = size + float(c["slopes"][h]) * (kp - qpos).abs()
                s = float(c["sink"][h]) if c["sink"] is not None else -math.inf
                top = max(float(x.max()), s)
                e = torch.exp(x - top)
                p = e / (e.sum() + math.exp(s - top))
                out[t, h] = p @ v
                A = p @ v.abs()
                # (weights that matter are within a few units of the largest score)
                w = (D + 8) * 2.0 ** -24 * float(((size + x.abs()) * p).max() + size[p > 1e-6].max()) + 2.0 ** -21
                tol[t, h] = u * (A + out[t, h].abs()) + 2 * w * A
                if dtype == torch.float16:
                    tol[t, h] += len(kp) * 2.0 ** -25 * v.abs().amax(0)
    return out, tol


def attention_by_sequence(c):
    """attention() with a sequence's rows and keys at once, for long contexts."""
    H, Hk, D, bs, dtype = c["H"], c["Hk"], c["D"], c["bs"], c["dtype"]
    u, G = HALF_STEP[dtype], c["H"] // c["Hk"]
    scale = c["scale"] or 1 / math.sqrt(D)
    out, tol = torch.zeros(c["T"], H, D).double(), torch.zeros(c["T"], H, D).double()
    for b in range(c["B"]):
        past, n, t0 = c["past"][b], c["n"][b], int(c["cum"][b])
        p = torch.arange(past + n)
        blocks = c["table"][b].long()[p // bs]
        p, slots = p[blocks >= 0], (blocks * bs + p % bs)[blocks >= 0]
        if n == 0 or p.numel() == 0:
            continue
        rows = slice(t0, t0 + n)
        node = p - past
        draft = node.clamp(min=0)
        qpos = c["pos"][rows].long() if c["positions"] is not None else past + torch.arange(n)
        kpos = torch.where(node >= 0, qpos[draft], p)
        see = torch.where(node >= 0, c["rows"][rows][:, draft], torch.ones(n, 1, dtype=torch.bool))
        if c["window"] > 0:
            see = see & (kpos > qpos.clamp(min=past)[:, None] - c["window"])
        gap = (kpos - qpos[:, None]).double()
        for k in range(Hk):
            heads = slice(k * G, (k + 1) * G)
            q = c["query"].view(c["T"], H, D)[rows, heads].double()
            K, V = (c[name].view(-1, Hk, D)[slots, k].double() for name in ("key_cache", "value_cache"))
            x, size = q @ K.T * scale, q.abs() @ K.abs().T * scale  # [n, G, keys]
            if c["softcap"]:
                x, size = c["softcap"] * torch.tanh(x / c["softcap"]), size + 2 * c["softcap"]
            if c["slopes"] is not None:
                bias = c["slopes"][heads].double()[:, None] * gap[:, None]
                x, size = x + bias, size + bias.abs()
            x = torch.where(see[:, None], x, -math.inf)
            s = c["sink"][heads].double()[:, None] if c["sink"] is not None else torch.full((G, 1), -math.inf).double()
            top = torch.maximum(x.amax(-1, keepdim=True), s)
            live = see.any(-1)[:, None, None].expand(n, G, 1)
            top = torch.where(live, top, 0.0)
            e = torch.exp(x - top)
            w8 = e / (e.sum(-1, keepdim=True) + torch.exp(s - top)).clamp(min=1e-300)
            o, A = w8 @ V, w8 @ V.abs()
            gone = torch.where(see[:, None], (size + x.abs()) * w8, 0.0).amax(-1, keepdim=True)
            most = torch.where(w8 > 1e-6, size, 0.0).amax(-1, keepdim=True)
            w = (D + 8) * 2.0 ** -24 * (gone + most) + 2.0 ** -21
            t = u * (A + o.abs()) + 2 * w * A
            if dtype == torch.float16:
                t = t + see.sum(-1)[:, None, None] * 2.0 ** -25 * V.abs().amax(0)
            out[rows, heads] = torch.where(live, o, 0.0)
            tol[rows, heads] = torch.where(live, t, 0.0)
    return out, tol
