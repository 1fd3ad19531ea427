"""Measured cases of the operators that read a codebook back and train on its labels.

km_matvec4         products with weights held as 4-bit codes of per-row codebooks, with group scales
km_lookup          rows of a table for a vector of ids, scaled
km_lookup_grad     the table's gradient: the output's gradient summed over the tokens of each id
km_xent            softmax cross entropy of points against all K table rows, without the N x K logits
km_xent_grad       its gradient with respect to the points and the table

`run` computes them in plain torch (32 bits, rounded once) where `own` is false, and calls the
library where it is true. `exact` evaluates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one 4096 x 4096 weight matrix with a 16-value codebook per row (the row-codebook fits of
        # this library), one token: the product of a single decoding step, bound by latency
        {"name": "matvec4_row_codebooks", "op": "matvec4", "R": 4096, "N": 4096, "M": 1, "K": 16, "group": 0, "dtype": "f16"},
        # a wide projection with a scale per 128 weights, one token: bound by the codes' bytes
        {"name": "matvec4_wide_groups", "op": "matvec4", "R": 32768, "N": 8192, "M": 1, "K": 16, "group": 128, "dtype": "bf16"},
        # sixteen sequences decoded together, a scale per 64 weights
        {"name": "matvec4_16_tokens", "op": "matvec4", "R": 8192, "N": 8192, "M": 16, "K": 16, "group": 64, "dtype": "bf16"},
        # odd sizes, fp32 tokens, 8-value codebooks
        {"name": "matvec4_ragged_f32", "op": "matvec4", "R": 1003, "N": 1999, "M": 3, "K": 8, "group": 0, "dtype": "f32"},
        # the table rows of one short prompt: the smallest call
        {"name": "lookup_prompt", "op": "lookup", "B": 1, "N": 100, "K": 8192, "d": 1024, "dtype": "bf16"},
        # a batch of vector-quantised points read back: the labels of the batched assignment
        {"name": "lookup_decode", "op": "lookup", "B": 32, "N": 65536, "K": 1024, "d": 128, "dtype": "f16"},
        # one training step's token gradient: many more rows than any step touches, Zipf ids
        {"name": "lookup_grad_tokens", "op": "lookup_grad", "B": 1, "N": 16384, "K": 65536, "d": 1024, "dtype": "bf16", "out": "bf16"},
        # the codebook's gradient of a batch of quantised points: every row many times
        {"name": "lookup_grad_clusters", "op": "lookup_grad", "B": 32, "N": 65536, "K": 1024, "d": 128, "dtype": "f16", "out": "f32"},
        # the loss of one short, odd sequence over a small codebook
        {"name": "xent_small", "op": "xent", "B": 1, "N": 257, "K": 1000, "d": 128, "dtype": "f16"},
        # the loss of a batch of tokens over a large vocabulary
        {"name": "xent_vocabulary", "op": "xent", "B": 1, "N": 8192, "K": 32768, "d": 1024, "dtype": "bf16"},
        # the same as a training step: loss and both gradients
        {"name": "xent_train_vocabulary", "op": "xent_train", "B": 1, "N": 8192, "K": 32768, "d": 1024, "dtype": "bf16"},
        # training on the labels of the large-K assignment: K = 8192 at d = 128
        {"name": "xent_train_labels", "op": "xent_train", "B": 1, "N": 32768, "K": 8192, "d": 128, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec4", "lookup", "lookup_grad", "xent", "xent_train"])
    if op == "matvec4":
        while True:
            c = {"op": op, "R": _log(rng, 64, 32768), "N": _log(rng, 64, 16384), "M": rng.choice([1, 1, 1, _log(rng, 2, 32)]),
                 "K": rng.choice([2, 8, 15, 16, 16, 16]), "group": rng.choice([0, 32, 64, 128, 256]),
                 "dtype": rng.choice(["f16", "bf16", "bf16", "f32"])}
            if c["R"] * c["N"] <= 32768 * 8192:
                return c
    if op == "lookup":
        while True:
            c = {"op": op, "B": rng.choice([1, 1, 2, 8, 32]), "N": _log(rng, 1, 65536), "K": _log(rng, 2, 131072),
                 "d": rng.choice([_log(rng, 1, 4096), 8 * _log(rng, 1, 512)]), "dtype": rng.choice(["f16", "bf16", "f32"])}
            if c["B"] * c["N"] * c["d"] <= 1 << 28 and c["B"] * c["K"] * c["d"] <= 1 << 28:
                return c
    if op == "lookup_grad":
        while True:
            c = {"op": op, "B": rng.choice([1, 1, 2, 8, 32]), "N": _log(rng, 1, 65536), "K": _log(rng, 2, 131072),
                 "d": rng.choice([_log(rng, 1, 4096), 8 * _log(rng, 1, 512)]), "dtype": rng.choice(["f16", "bf16", "f32"])}
            c["out"] = rng.choice([c["dtype"], "f32"])
            if c["B"] * c["N"] * c["d"] <= 1 << 28 and c["B"] * c["K"] * c["d"] <= 1 << 27:
                return c
    while True:
        c = {"op": op, "B": rng.choice([1, 1, 1, 2, 4]), "N": _log(rng, 1, 32768), "K": _log(rng, 2, 65536),
             "d": rng.choice([_log(rng, 1, 2048), 8 * _log(rng, 4, 256)]), "dtype": rng.choice(["f16", "bf16"])}
        if c["B"] * c["N"] * c["K"] <= 1 << 28 and c["B"] * c["N"] * c["K"] * c["d"] <= 1 << 38:
            return c


# ------------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] == "matvec4":
        R, N, M, K, group = (case[k] for k in ("R", "N", "M", "K", "group"))
        codes = torch.randint(0, K, (R, N), generator=g, device=dev, dtype=torch.uint8)
        s["packed"] = _pack(codes)
        # fitted codebooks are sorted, a few hundredths wide (Student-t rows times 0.02); with
        # group scales they cover the normalised range instead
        s["C"] = (randn(R, K) * (0.5 if group else 0.02)).sort(1).values.contiguous()
        s["scales"] = (0.02 + 0.05 * torch.rand((R, -(-N // group)), generator=g, device=dev)) if group else None
        s["x"] = randn(M, N).to(dt)
        return s
    B, N, K, d = (case[k] for k in ("B", "N", "K", "d"))
    ids = _zipf(B, N, K, g, dev) if case["op"] in ("lookup", "lookup_grad") and K > 4096 else \
        torch.randint(0, K, (B, N), generator=g, device=dev, dtype=torch.int32)
    if N >= 64:
        # one token in 64 carries no label (padding)
        ids = torch.where(torch.rand((B, N), generator=g, device=dev) < 1 / 64, torch.full_like(ids, -1), ids)
    s["ids"] = ids.contiguous()
    if case["op"] == "lookup":
        s["C"], s["scale"] = randn(B, K, d).to(dt), float(np.float32(math.sqrt(d)))
    elif case["op"] == "lookup_grad":
        s["dY"], s["scale"] = randn(B, N, d).to(dt), float(np.float32(math.sqrt(d)))
    else:
        # logits of a few units: unit points against rows of size 2 / sqrt(d), the label's row
        # partly aligned with its point as after some training
        s["C"] = (randn(B, K, d) * (2 / math.sqrt(d))).to(dt)
        pull = torch.gather(s["C"], 1, s["ids"].clamp(min=0).long()[..., None].expand(B, N, d))
        s["X"] = (randn(B, N, d) + 0.5 * pull.float()).to(dt)
        s["scale"] = 1.0
        # the mean's gradient; fp16 training scales its loss so that small gradients keep their bits
        s["g"] = torch.full((B, N), (1024.0 if dt == torch.float16 else 1.0) / (B * N), device=dev)
    return s


def _pack(codes):
    """Two codes per byte, the even position in the low half, rows padded to 16 bytes."""
    R, N = codes.shape
    full = torch.zeros((R, 32 * (-(-N // 32))), dtype=torch.uint8, device=codes.device)
    full[:, :N] = codes
    return (full[:, 0::2] | (full[:, 1::2] << 4)).contiguous()


def _zipf(B, N, K, g, dev):
    """Ids with frequencies ~ 1 / rank^1.1, ranks scattered over the table."""
    p = torch.arange(1, K + 1, device=dev, dtype=torch.float64).pow(-1.1)
    cdf = torch.cumsum(p / p.sum(), 0)
    u = torch.rand((B, N), generator=g, device=dev, dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp(max=K - 1)
    perm = torch.randperm(K, generator=g, device=dev)
    return perm[rank].to(torch.int32)


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import exact_lloyd_means_assign_b200 as km
        if op == "matvec4":
            return km.km_matvec4(s["x"], s["packed"], s["C"], s["scales"], s["case"]["group"])
        if op == "lookup":
            return km.km_lookup(s["C"], s["ids"], s["scale"])
        if op == "lookup_grad":
            return km.km_lookup_grad(s["dY"], s["ids"], s["case"]["K"], s["scale"], out_dtype=DT[s["case"]["out"]])
        loss, lse = km.km_xent(s["X"], s["C"], s["ids"], s["scale"])
        if op == "xent":
            return loss, lse
        dX, dC = km.km_xent_grad(s["X"], s["C"], s["ids"], lse, s["g"], s["scale"])
        return loss, lse, dX, dC
    return {"matvec4": _matvec4, "lookup": _lookup, "lookup_grad": _lookup_grad, "xent": _xent, "xent_train": _xent_train}[op](s)


def _matvec4(s):
    x, dt, N = s["x"], s["x"].dtype, s["x"].shape[1]
    packed = s["packed"]
    codes = torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1)[:, :N]
    W = torch.gather(s["C"].to(dt).float(), 1, codes.long())  # values rounded to the tokens' type
    if s["scales"] is not None:
        W = W * s["scales"].repeat_interleave(s["case"]["group"], 1)[:, :N]
    return (x.float() @ W.t()).to(dt)


def _lookup(s):
    C, ids = s["C"], s["ids"]
    rows = ids.clamp(min=0).long() + torch.arange(C.shape[0], device=C.device)[:, None] * C.shape[1]
    y = C.flatten(0, 1)[rows].float() * s["scale"]
    return torch.where((ids >= 0)[..., None], y, torch.zeros((), device=C.device)).to(C.dtype)


def _lookup_grad(s):
    dY, ids, K = s["dY"], s["ids"], s["case"]["K"]
    B, N, d = dY.shape
    rows = torch.where(ids >= 0, ids.long() + torch.arange(B, device=ids.device)[:, None] * K, B * K)
    out = torch.zeros((B * K + 1, d), device=dY.device)
    out.index_add_(0, rows.flatten(), dY.flatten(0, 1).float())
    return (out[:-1].view(B, K, d) * s["scale"]).to(DT[s["case"]["out"]])


def _xent_parts(s):
    X, C, ids = s["X"].float(), s["C"].float(), s["ids"]
    z = torch.bmm(X, C.transpose(1, 2)) * s["scale"]
    m = z.amax(2, keepdim=True)
    e = torch.exp(z - m)
    tot = e.sum(2, keepdim=True)
    lse = (m + torch.log(tot)).squeeze(2)
    zt = torch.gather(z, 2, ids.clamp(min=0).long()[..., None]).squeeze(2)
    loss = torch.where(ids >= 0, lse - zt, torch.zeros((), device=z.device))
    return X, C, ids, e, tot, loss, lse


def _xent(s):
    *_, loss, lse = _xent_parts(s)
    return loss, lse


def _xent_train(s):
    X, C, ids, e, tot, loss, lse = _xent_parts(s)
    w = torch.where(ids >= 0, s["g"] * s["scale"], torch.zeros((), device=X.device))[..., None]
    P = e / tot * w
    P.scatter_add_(2, ids.clamp(min=0).long()[..., None], -w)
    dt = s["X"].dtype
    return loss, lse, torch.bmm(P, C).to(dt), torch.bmm(P.transpose(1, 2), X).to(dt)


# ------------------------------------------------------------------------------------ the work

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "matvec4":
        R, N, M, K, group = (case[k] for k in ("R", "N", "M", "K", "group"))
        sc = R * -(-N // group) * 4 if group else 0
        return {"bytes": R * N / 2 + R * K * 4 + sc + M * N * es + M * R * es, "flops": 2.0 * M * R * N}
    B, N, K, d = (case[k] for k in ("B", "N", "K", "d"))
    if case["op"] == "lookup":
        # a table row that several tokens name is read once
        return {"bytes": B * (N * d * es + min(N, K) * d * es + N * 4), "flops": float(B * N * d)}
    if case["op"] == "lookup_grad":
        eo = 4 if case["out"] == "f32" else 2
        return {"bytes": B * (N * d * es + K * d * eo + N * 4), "flops": float(B * N * d)}
    train = case["op"] == "xent_train"
    nbytes = B * ((N + K) * d * es * (2 if train else 1) + N * (16 if train else 12))
    # one product for the logits, one for each gradient
    return {"bytes": nbytes, "flops": 2.0 * B * N * K * d * (3 if train else 1)}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec4":
        x, K, N = s["x"].double(), case["K"], case["N"]
        Cr = s["C"].to(s["x"].dtype).double()
        y = torch.zeros((x.shape[0], case["R"]), dtype=torch.float64, device=x.device)
        step = max(1, (1 << 27) // N)
        for r in range(0, case["R"], step):
            p = s["packed"][r:r + step].int()
            codes = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=torch.int32, device=p.device)
            codes[:, 0::2] = p % 16
            codes[:, 1::2] = p // 16
            codes = codes[:, :N]
            if s["scales"] is None:
                xs = [(slice(0, N), torch.ones((p.shape[0], 1), dtype=torch.float64, device=x.device))]
            else:
                G = case["group"]
                xs = [(slice(i, min(N, i + G)), s["scales"][r:r + step, i // G, None].double()) for i in range(0, N, G)]
            if len(xs) > 1:
                W = torch.zeros((p.shape[0], N), dtype=torch.float64, device=x.device)
                for k in range(K):
                    W += (codes == k) * Cr[r:r + step, k, None]
                for sl, sc in xs:
                    W[:, sl] *= sc
                y[:, r:r + step] = torch.einsum("mn,rn->mr", x, W)
            else:
                # sum over the K values of the value times the sum of the tokens that carry its code
                for k in range(K):
                    y[:, r:r + step] += Cr[r:r + step, k] * torch.einsum("mn,rn->mr", x, (codes == k).double())
        return y
    ids = s["ids"].long()
    B, N, K, d = (case[k] for k in ("B", "N", "K", "d"))
    dev = ids.device
    if case["op"] == "lookup":
        y = torch.zeros((B, N, d), dtype=torch.float64, device=dev)
        for b in range(B):
            ok = ids[b] >= 0
            y[b, ok] = s["scale"] * s["C"][b].double().index_select(0, ids[b][ok])
        return y
    if case["op"] == "lookup_grad":
        out = torch.zeros((B, K, d), dtype=torch.float64, device=dev)
        for b in range(B):
            ok = ids[b] >= 0
            out[b].index_put_((ids[b][ok],), s["dY"][b][ok].double() * s["scale"], accumulate=True)
        return out
    X, C = s["X"].double(), s["C"].double()
    train = case["op"] == "xent_train"
    loss = torch.zeros((B, N), dtype=torch.float64, device=dev)
    lse = torch.zeros((B, N), dtype=torch.float64, device=dev)
    dX, dC = torch.zeros_like(X), torch.zeros_like(C)
    step = max(1, (1 << 27) // K)
    for b in range(B):
        for n in range(0, N, step):
            sl = slice(n, n + step)
            z = s["scale"] * torch.einsum("nd,kd->nk", X[b, sl], C[b])
            lse[b, sl] = torch.logsumexp(z, 1)
            ok = (ids[b, sl] >= 0).nonzero().squeeze(1)
            t = ids[b, sl][ok]
            loss[b, n + ok] = lse[b, sl][ok] - z[ok, t]
            if train:
                p = torch.softmax(z, 1)
                p[ok, t] -= 1
                w = torch.zeros(p.shape[0], dtype=torch.float64, device=dev)
                w[ok] = s["g"][b, sl][ok].double() * s["scale"]
                p *= w[:, None]
                dX[b, sl] = torch.einsum("nk,kd->nd", p, C[b])
                dC[b] += torch.einsum("nk,nd->kd", p, X[b, sl])
    return (loss, lse, dX, dC) if train else (loss, lse)
