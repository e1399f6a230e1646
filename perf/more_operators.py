"""The operators at the two ends of a language model and between its products, as cases to measure.

Seven kinds of pass, each the calls that a user's program makes of the package's binding:

  embed          token ids to scaled rows of the embedding table
  embed_back     the table's whole gradient from the rows' gradients
  qk             RMS norm of every query and key head, then the rotation of its position
  qk_back        its gradients (heads and both norm weights)
  logprobs       log probabilities of given tokens, entropy, the most probable tokens
  logprobs_back  the logits' gradient from those of log probability and entropy
  clip           the global norm of a model's gradients, and the gradients clipped to it

``run`` computes a pass in elementary torch operations in FP32, or, with
``own`` set, through the package.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases --

def listed():
    return [
        # one decode step of eight sequences, hidden size 8192: latency
        dict(name="embed_decode_8x8192", kind="embed", tokens=8, K=8192, vocab=128256, dtype="bf16", scaled=False,
             padded=False),
        # a long prefill, rows scaled by the root of the hidden size, padding behind the last sequence
        dict(name="embed_prefill_16384x8192", kind="embed", tokens=16384, K=8192, vocab=128256, dtype="bf16",
             scaled=True, padded=True),
        # a training step's gradient of a large table: few of its rows occur, some of them thousands of times
        dict(name="embed_back_32768x4096", kind="embed_back", tokens=32768, K=4096, vocab=128256, dtype="bf16",
             scaled=False, padded=True),
        # a short ragged batch trained in FP32 with a small vocabulary
        dict(name="embed_back_f32_1023x2048", kind="embed_back", tokens=1023, K=2048, vocab=32000, dtype="f32",
             scaled=True, padded=False),
        # decode batch of 32 sequences at far positions, 64 query and 8 key heads
        dict(name="qk_decode_32x72x128", kind="qk", tokens=32, q_heads=64, k_heads=8, D=128, rotary=128,
             positions=131072, dtype="bf16", norm=True, interleaved=False),
        # a long prefill of packed sequences, 32 query and 8 key heads inside the product's q|k|v rows
        dict(name="qk_prefill_16384x40x128", kind="qk", tokens=16384, q_heads=32, k_heads=8, D=128, rotary=128,
             positions=32768, dtype="bf16", norm=True, interleaved=False),
        # and the gradient of a training step
        dict(name="qk_back_8192x40x128", kind="qk_back", tokens=8192, q_heads=32, k_heads=8, D=128, rotary=128,
             positions=32768, dtype="bf16", norm=True, interleaved=False),
        # sampling for sixteen sequences with the twenty most probable tokens reported, temperature 0.7
        dict(name="logprobs_decode_16x128256", kind="logprobs", rows=16, vocab=128256, dtype="bf16", top=20,
             scale=1 / 0.7, masked=False),
        # scoring a ragged batch in FP32 with a vocabulary of odd size, so that rows start on any 4-byte boundary
        dict(name="logprobs_score_f32_1023x50257", kind="logprobs", rows=1023, vocab=50257, dtype="f32", top=5,
             scale=1.0, masked=False),
        # the loss's gradient of a training step, with a bonus for entropy
        dict(name="logprobs_back_4096x128256", kind="logprobs_back", rows=4096, vocab=128256, dtype="bf16",
             scale=1.0, entropy=True),
        # low-rank adapters of all products of 32 layers: hundreds of small FP32 gradients
        dict(name="clip_adapters_448", kind="clip", layout="adapters", layers=32, hidden=4096, inner=14336,
             dtype="f32", out="f32"),
        # four full layers' gradients, clipped into the FP32 buffer that the optimizer reads
        dict(name="clip_layers_4", kind="clip", layout="layers", layers=4, hidden=4096, inner=14336, dtype="bf16",
             out="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["embed", "embed_back", "qk", "qk_back", "logprobs", "logprobs_back", "clip"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    e = 2 if dtype == "bf16" else 4
    c = dict(kind=kind, dtype=dtype)
    if kind in ("embed", "embed_back"):
        K = 32 * _spread(rng, 8, 256)
        vocab = _spread(rng, 1000, min(262144, 1_000_000_000 // (e * K)))
        tokens = _spread(rng, 1, min(32768, 270_000_000 // (e * K)))
        c.update(tokens=tokens, K=K, vocab=vocab, scaled=rng.random() < 0.5, padded=rng.random() < 0.5)
    elif kind in ("qk", "qk_back"):
        D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        k_heads = rng.choice([1, 2, 4, 8, 8, 16])
        q_heads = k_heads * rng.randrange(1, 9)
        tokens = _spread(rng, 1, min(16384, 160_000_000 // (e * D * (q_heads + k_heads))))
        rotary = rng.choice([D, D, D, D // 32 * 16])
        c.update(tokens=tokens, q_heads=q_heads, k_heads=k_heads, D=D, rotary=rotary,
                 positions=_spread(rng, 2048, 131072), norm=rng.random() < 0.7, interleaved=rng.random() < 0.3)
    elif kind in ("logprobs", "logprobs_back"):
        vocab = _spread(rng, 500, 262144)
        scale = rng.choice([1.0, 1.0, 1 / 0.7, 0.5])
        if kind == "logprobs":
            top = rng.choice([0, 0, 1, 5, 20])
            rows = _spread(rng, 1, min(8192, (250_000_000 if top else 1_000_000_000) // (e * vocab)))
            c.update(rows=rows, vocab=vocab, top=top, scale=scale, masked=rng.random() < 0.3)
        else:
            rows = _spread(rng, 1, min(8192, 900_000_000 // (e * vocab)))
            c.update(rows=rows, vocab=vocab, scale=scale, entropy=rng.random() < 0.5)
    else:
        layout = rng.choice(["adapters", "layers"])
        hidden, inner = 128 * _spread(rng, 4, 32), 128 * _spread(rng, 8, 112)
        most = 48 if layout == "adapters" else max(1, min(32, 400_000_000 // (hidden * (3 * hidden + 3 * inner))))
        c.update(layout=layout, layers=rng.randrange(1, most + 1), hidden=hidden, inner=inner,
                 out=rng.choice([dtype, "f32"]))
    return c


def _grad_shapes(c):
    """Shapes of the gradients, in the order of the parameters."""
    H, F = c["hidden"], c["inner"]
    products = [(H, H), (H // 4, H), (H // 4, H), (H, H), (F, H), (F, H), (H, F)]
    if c["layout"] == "adapters":
        return [s for _ in range(c["layers"]) for n, k in products for s in ((16, k), (n, 16))]
    return [s for _ in range(c["layers"]) for s in products + [(H,), (H,)]]


def _zipf(vocab):
    """The share of each rank among tokens."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _real_tokens(c):
    return c["tokens"] - c["tokens"] // 16 if c["padded"] else c["tokens"]


# ---------------------------------------------------------------- their work --

def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["kind"] in ("embed", "embed_back"):
        rows = float((1.0 - (1.0 - _zipf(c["vocab"])) ** _real_tokens(c)).sum())  # different ids that are expected
        if c["kind"] == "embed":
            return {"bytes": e * c["K"] * (rows + c["tokens"]) + 8 * c["tokens"], "flops": c["tokens"] * c["K"]}
        return {"bytes": e * c["K"] * (_real_tokens(c) + c["vocab"]) + 8 * c["tokens"],
                "flops": _real_tokens(c) * c["K"]}
    if c["kind"] in ("qk", "qk_back"):
        heads = c["tokens"] * (c["q_heads"] + c["k_heads"])
        n, angles = heads * c["D"], 4 * min(c["tokens"], c["positions"]) * c["rotary"] + 8 * c["tokens"]
        weights = 2 * e * c["D"] if c["norm"] else 0
        if c["kind"] == "qk":
            return {"bytes": 2 * e * n + angles + weights + (4 * heads if c["norm"] else 0), "flops": 9 * n}
        extra = e * n + 4 * heads + weights + 8 * c["D"] if c["norm"] else 0
        return {"bytes": 2 * e * n + angles + extra, "flops": 13 * n}
    if c["kind"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": e * n + c["rows"] * (8 + 16 + 12 * c["top"]), "flops": 6 * n}
    if c["kind"] == "logprobs_back":
        n = c["rows"] * c["vocab"]
        return {"bytes": 2 * e * n + c["rows"] * (8 + 12 + (8 if c["entropy"] else 0)), "flops": 6 * n}
    n = sum(math.prod(s) for s in _grad_shapes(c))
    return {"bytes": n * (e + (2 if c["out"] == "bf16" else 4)) + 4, "flops": 3 * n}


# -------------------------------------------------------------------- inputs --

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _uniform(gen, n):
    return torch.rand((n,), generator=gen, device=DEV, dtype=torch.float64)


def _token_ids(gen, c):
    """Ids of a text: a few very frequent, most rare, spread over the vocabulary; padding (-1) behind the last one."""
    share = torch.from_numpy(np.cumsum(_zipf(c["vocab"]))).to(DEV)
    rank = torch.searchsorted(share, _uniform(gen, c["tokens"])).clamp(max=c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=gen, device=DEV)[rank]
    ids[_real_tokens(c):] = -1
    return ids


def _angles(c):
    """cos | sin [positions, rotary] of position * 10000^(-2i / rotary), formed in 64 bits."""
    half = c["rotary"] // 2
    freq = torch.pow(10000.0, -torch.arange(half, device=DEV, dtype=torch.float64) / half)
    a = torch.arange(c["positions"], device=DEV, dtype=torch.float64).unsqueeze(1) * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _logits(gen, rows, vocab, dtype):
    """A model's logits: a broad body, and for most rows a few tokens that stand out."""
    x = torch.randn((rows, vocab), generator=gen, device=DEV, dtype=torch.float32).mul_(2.0)
    at = torch.randint(0, vocab, (rows, min(8, vocab)), generator=gen, device=DEV)
    x.scatter_add_(1, at, 8.0 * torch.rand(at.shape, generator=gen, device=DEV) + 2.0)
    return x.to(dtype), at


def _row_statistics(x, scale, entropy):
    """(max, log of the sum relative to it) of every row, and its entropy, from 64 bits, a few rows at a time."""
    stats, ent = [], []
    for part in x.split(256):
        z = part.double()
        m = z.amax(1, keepdim=True)
        z = (z - m) * scale
        s = torch.logsumexp(z, 1, keepdim=True)
        stats.append(torch.cat([m, s], 1).float())
        if entropy:
            z = z - s
            ent.append(-(z.exp() * z).sum(1).float())
    return torch.cat(stats), torch.cat(ent) if entropy else None


def prepare(case, seed):
    c, dt = case, _dtype(case["dtype"])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["kind"] in ("embed", "embed_back"):
        s["ids"] = _token_ids(gen, c)
        s["scale"] = math.sqrt(c["K"]) if c["scaled"] else 1.0
        if c["kind"] == "embed":
            s["table"] = _normal(gen, (c["vocab"], c["K"]), dt, 0.02)
            s["out"] = torch.empty((c["tokens"], c["K"]), dtype=dt, device=DEV)
        else:
            s["dy"] = _normal(gen, (c["tokens"], c["K"]), dt, 0.02)
            s["dtable"] = torch.empty((c["vocab"], c["K"]), dtype=dt, device=DEV)
    elif c["kind"] in ("qk", "qk_back"):
        T, H, D = c["tokens"], c["q_heads"] + c["k_heads"], c["D"]
        qkv = _normal(gen, (T, H + c["k_heads"], D), dt, 1.5)
        s["x"] = qkv[:, :H]  # queries and keys inside the rows that the product left
        s["rope"] = _angles(c)
        # packed sequences: positions count on from a start of their own
        starts = torch.randint(0, T, (max(1, T // 1500),), generator=gen, device=DEV).sort().values
        first = torch.randint(0, c["positions"], (starts.numel() + 1,), generator=gen, device=DEV)
        t = torch.arange(T, device=DEV)
        s["positions"] = (first[torch.searchsorted(starts, t, right=True)] + t) % c["positions"]
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = (1.0 + 0.2 * torch.randn((D,), generator=gen, device=DEV)).to(dt)
            s["kw"] = (1.0 + 0.2 * torch.randn((D,), generator=gen, device=DEV)).to(dt)
        if c["kind"] == "qk":
            s["y"] = torch.empty((T, H, D), dtype=dt, device=DEV)
            s["rstd"] = torch.empty((T, H), dtype=torch.float32, device=DEV) if c["norm"] else None
        else:
            s["dy"] = _normal(gen, (T, H, D), dt, 0.02)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(2) + 1e-6) if c["norm"] else None
            s["dx"] = torch.empty((T, H, D), dtype=dt, device=DEV)
            s["dqw"] = torch.empty((D,), dtype=torch.float32, device=DEV) if c["norm"] else None
            s["dkw"] = torch.empty((D,), dtype=torch.float32, device=DEV) if c["norm"] else None
    elif c["kind"] in ("logprobs", "logprobs_back"):
        rows, V = c["rows"], c["vocab"]
        s["x"], at = _logits(gen, rows, V, dt)
        s["targets"] = at[:, 0].contiguous()
        f32 = dict(dtype=torch.float32, device=DEV)
        if c["kind"] == "logprobs":
            if c["masked"]:  # a third of the rows allow a few tokens only, as under a grammar, or most
                allowed = torch.rand((rows, V), generator=gen, device=DEV) < torch.where(
                    torch.arange(rows, device=DEV) % 2 == 0, 0.002, 0.7).unsqueeze(1)
                allowed.scatter_(1, s["targets"].unsqueeze(1), True)
                allowed |= (torch.arange(rows, device=DEV) % 3 != 0).unsqueeze(1)
                s["x"].masked_fill_(~allowed, float("-inf"))
                del allowed
            s["logprob"], s["entropy"] = torch.empty((rows,), **f32), torch.empty((rows,), **f32)
            s["stats"] = torch.empty((rows, 2), **f32)
            s["top_ids"] = torch.empty((rows, c["top"]), dtype=torch.int64, device=DEV) if c["top"] else None
            s["top_logprobs"] = torch.empty((rows, c["top"]), **f32) if c["top"] else None
        else:
            s["targets"][rows // 2:rows // 2 + rows // 20] = -100  # a prompt's tokens do not count
            s["stats"], s["entropy"] = _row_statistics(s["x"], c["scale"], c["entropy"])
            s["dlogprob"] = _normal(gen, (rows,), torch.float32, 1.0)
            s["dentropy"] = _normal(gen, (rows,), torch.float32, 0.1) if c["entropy"] else None
            s["dlogits"] = torch.empty((rows, V), dtype=dt, device=DEV)
    else:
        sizes = random.Random(seed)
        s["grads"] = [_normal(gen, shape, dt, 10.0 ** sizes.uniform(-4, -2)) for shape in _grad_shapes(c)]
        n = [g.numel() for g in s["grads"]]
        s["flat"] = torch.empty((sum(n),), dtype=_dtype(c["out"]), device=DEV)
        s["out"] = [f.view(g.shape) for f, g in zip(s["flat"].split(n), s["grads"])]
        s["max_norm"] = 0.5
    return s


# ------------------------------------------------------------ the plain form --

def _turn(x, cos, sin, rotary, interleaved):
    """The first `rotary` values of every head, turned in pairs by the angles' cosines and sines."""
    head, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = head[..., :rotary // 2], head[..., rotary // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _run_plain(s):
    c, dt = s["case"], _dtype(s["case"]["dtype"])
    if c["kind"] == "embed":
        real = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        rows = s["table"][torch.where(real, s["ids"], 0)].float() * s["scale"]
        return {"out": torch.where(real.unsqueeze(1), rows, 0.0).to(dt)}
    if c["kind"] == "embed_back":
        real = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
        dtable = torch.zeros((c["vocab"], c["K"]), dtype=torch.float32, device=DEV)
        dtable.index_add_(0, s["ids"][real], s["dy"].float()[real])
        return {"dtable": (dtable * s["scale"]).to(dt)}
    if c["kind"] in ("qk", "qk_back"):
        angles = s["rope"][s["positions"]].unsqueeze(1)
        cos, sin = angles[..., :c["rotary"] // 2], angles[..., c["rotary"] // 2:]
        x = s["x"].float()
        w = None
        if c["norm"]:
            w = torch.cat([s["qw"].float().expand(c["q_heads"], -1), s["kw"].float().expand(c["k_heads"], -1)])
        if c["kind"] == "qk":
            rstd = None
            if c["norm"]:
                rstd = torch.rsqrt(x.square().mean(2) + 1e-6)
                x = x * rstd.unsqueeze(2) * w
            return {"y": _turn(x, cos, sin, c["rotary"], c["interleaved"]).to(dt), "rstd": rstd}
        dy = _turn(s["dy"].float(), cos, -sin, c["rotary"], c["interleaved"])
        if not c["norm"]:
            return {"dx": dy.to(dt), "dqw": None, "dkw": None}
        n, p = x * s["rstd"].unsqueeze(2), dy * w
        dw = (dy * n).sum(0)
        dx = (p - n * (p * n).mean(2, keepdim=True)) * s["rstd"].unsqueeze(2)
        return {"dx": dx.to(dt), "dqw": dw[:c["q_heads"]].sum(0), "dkw": dw[c["q_heads"]:].sum(0)}
    if c["kind"] in ("logprobs", "logprobs_back"):
        x = s["x"].float()
        real = (s["targets"] >= 0) & (s["targets"] < c["vocab"])
        at = torch.where(real, s["targets"], 0).unsqueeze(1)
        if c["kind"] == "logprobs":
            m = x.amax(1, keepdim=True)
            z = (x - m) * c["scale"]
            e = z.exp()
            total = e.sum(1, keepdim=True)
            log_total = total.log()
            entropy = log_total - torch.where(e > 0, e * z, 0.0).sum(1, keepdim=True) / total
            logprob = torch.where(real, (z.gather(1, at) - log_total).squeeze(1), 0.0)
            out = {"logprob": logprob, "entropy": entropy.squeeze(1), "stats": torch.cat([m, log_total], 1)}
            if c["top"]:
                del e
                ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
                z = z.gather(1, ids)
                out["top_ids"] = torch.where(z > float("-inf"), ids, -1)
                out["top_logprobs"] = z - log_total
            return out
        logp = (x - s["stats"][:, :1]) * c["scale"] - s["stats"][:, 1:]
        p = logp.exp()
        g = torch.where(real, s["dlogprob"], 0.0).unsqueeze(1)
        d = p * -g
        if s["dentropy"] is not None:
            d = d - torch.where(p > 0, p * (logp + s["entropy"].unsqueeze(1)), 0.0) * s["dentropy"].unsqueeze(1)
        d.scatter_add_(1, at, g)
        return {"dlogits": (d * c["scale"]).to(dt)}
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    out = torch.cat([(g.float() * factor).flatten() for g in s["grads"]]).to(_dtype(c["out"]))
    return {"norm": norm.float().reshape(1), "out": out}


# ----------------------------------------------------------- the package's --

def _run_own(s):
    from mx_block_scaled_gb300 import binding as mx
    c = s["case"]
    if c["kind"] == "embed":
        mx.embed(s["ids"], s["table"], scale=s["scale"], out=s["out"])
        return {"out": s["out"]}
    if c["kind"] == "embed_back":
        mx.embed_backward(s["dy"], s["ids"], c["vocab"], scale=s["scale"], dtable=s["dtable"])
        return {"dtable": s["dtable"]}
    if c["kind"] == "qk":
        mx.qk_norm_rope(s["x"], c["q_heads"], s["qw"], s["kw"], 1e-6, rope=s["rope"], positions=s["positions"],
                        interleaved=c["interleaved"], y=s["y"], rstd=s["rstd"])
        return {"y": s["y"], "rstd": s["rstd"]}
    if c["kind"] == "qk_back":
        mx.qk_norm_rope_backward(s["dy"], s["x"], s["rstd"], c["q_heads"], s["qw"], s["kw"], rope=s["rope"],
                                 positions=s["positions"], interleaved=c["interleaved"], dx=s["dx"],
                                 dq_weight=s["dqw"], dk_weight=s["dkw"])
        return {"dx": s["dx"], "dqw": s["dqw"], "dkw": s["dkw"]}
    if c["kind"] == "logprobs":
        mx.logprobs(s["x"], s["targets"], scale=c["scale"], top=c["top"], logprob=s["logprob"], entropy=s["entropy"],
                    stats=s["stats"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
        out = {"logprob": s["logprob"], "entropy": s["entropy"], "stats": s["stats"]}
        if c["top"]:
            out.update(top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
        return out
    if c["kind"] == "logprobs_back":
        mx.logprobs_backward(s["x"], s["targets"], s["stats"], s["dlogprob"], entropy=s["entropy"],
                             dentropy=s["dentropy"], scale=c["scale"], dlogits=s["dlogits"])
        return {"dlogits": s["dlogits"]}
    norm, _ = mx.clip_grads(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "out": s["flat"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------- the definition in 64 bits --

def _x_turn(x, a, b, cos, sin):
    """x with its values at index lists a and b turned in pairs."""
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "embed":
        out = torch.zeros((c["tokens"], c["K"]), dtype=torch.float64, device=DEV)
        at = torch.nonzero(s["ids"] >= 0).reshape(-1)
        out[at] = s["table"].double()[s["ids"][at]] * s["scale"]
        return {"out": out}
    if c["kind"] == "embed_back":
        # the rows' running sums in the order of the ids: an id's sum is a difference of two of them
        order = torch.argsort(s["ids"], stable=True)
        ids = s["ids"][order]
        order, ids = order[ids >= 0], ids[ids >= 0]
        dtable = torch.zeros((c["vocab"], c["K"]), dtype=torch.float64, device=DEV)
        found, count = torch.unique_consecutive(ids, return_counts=True)
        end = count.cumsum(0)
        for k in range(0, c["K"], 512):
            sums = torch.cat([dtable.new_zeros((1, min(512, c["K"] - k))),
                              s["dy"][order, k:k + 512].double().cumsum(0)])
            dtable[found, k:k + 512] = (sums[end] - sums[end - count]) * s["scale"]
        return {"dtable": dtable}
    if c["kind"] in ("qk", "qk_back"):
        half, D, Q = c["rotary"] // 2, c["D"], c["q_heads"]
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        angles = s["rope"].double()[s["positions"]][:, None]
        cos, sin = angles[..., :half], angles[..., half:]
        x = s["x"].double()
        if c["kind"] == "qk":
            rstd = None
            if c["norm"]:
                rstd = (x.pow(2).sum(2) / D + 1e-6).pow(-0.5)
                x = x * rstd[..., None]
                x = torch.cat([x[:, :Q] * s["qw"].double(), x[:, Q:] * s["kw"].double()], 1)
            return {"y": _x_turn(x, a, b, cos, sin), "rstd": rstd}
        dy = _x_turn(s["dy"].double(), b, a, cos, sin)  # back by the same angle
        if not c["norm"]:
            return {"dx": dy, "dqw": None, "dkw": None}
        r = s["rstd"].double()[..., None]
        p = torch.cat([dy[:, :Q] * s["qw"].double(), dy[:, Q:] * s["kw"].double()], 1)
        dx = r * p - r.pow(3) * x * ((p * x).sum(2, keepdim=True) / D)
        dw = dy * x * r
        return {"dx": dx, "dqw": dw[:, :Q].sum((0, 1)), "dkw": dw[:, Q:].sum((0, 1))}
    if c["kind"] == "logprobs":
        x = s["x"].double()
        lse = torch.logsumexp(x * c["scale"], 1)
        m = x.amax(1)
        logp = x * c["scale"] - lse[:, None]
        out = {"logprob": logp[torch.arange(c["rows"], device=DEV), s["targets"]],
               "entropy": torch.special.entr(logp.exp()).sum(1), "stats": torch.stack([m, lse - m * c["scale"]], 1)}
        if c["top"]:
            # by value, and among equal ones by place: both in one whole number, 32 bits each
            bits = s["x"].float().view(torch.int32).long()
            key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32
            key -= torch.arange(c["vocab"], device=DEV)
            at = torch.topk(key, min(c["top"], c["vocab"]), 1).indices
            top = logp.gather(1, at)
            out["top_ids"] = torch.where(torch.isinf(top), -1, at)
            out["top_logprobs"] = top
        return out
    if c["kind"] == "logprobs_back":
        out = torch.empty((c["rows"], c["vocab"]), dtype=torch.float64, device=DEV)
        for r in range(0, c["rows"], 512):
            part = slice(r, r + 512)
            t = s["targets"][part]
            logp = (s["x"][part].double() - s["stats"][part, :1].double()) * c["scale"] - s["stats"][part, 1:].double()
            p = logp.exp()
            g = torch.where(t >= 0, s["dlogprob"][part].double(), 0.0)[:, None]
            d = torch.where((torch.arange(c["vocab"], device=DEV) == t[:, None]), g, 0.0) - g * p
            if c["entropy"]:
                d += s["dentropy"][part, None].double() * (
                    torch.special.entr(p) - s["entropy"][part, None].double() * p)
            out[part] = d * c["scale"]
        return {"dlogits": out}
    flat = torch.cat([g.double().reshape(-1) for g in s["grads"]])
    norm = torch.linalg.vector_norm(flat)
    return {"norm": norm.reshape(1), "out": flat * min(1.0, s["max_norm"] / (float(norm) + 1e-6))}
