"""Measured cases of the mixture-of-experts form of an NVFP4 layer.

Rows are sorted by expert: expert e owns rows offsets[e] .. offsets[e + 1] - 1
of every matrix below, and its block scales start at the 128-row tile
offsets[e] // 128 + e.  Four kinds of pass, each in its plain form (elementary
torch operations in fp32) and as the calls that a program makes of this
package:

  route     the router: the k largest logits of each token, their softmax
            weights, and the rows that the chosen experts' products get
  quantize  rows to NVFP4 with one global scale per expert, and back to plain
            values: tokens fanned out to their experts' rows, or (gated) the
            activation between the experts' two products
  linear    the products grouped by expert, ragged sizes
  combine   the weighted sum of a token's rows, and what is added to it

Packed 4-bit codes are returned as the values they stand for, through the
package's way back: 16 bits where the quantized values are given, E4M3 where
they are computed (a last-place difference of the activation may move a code
by a step there).  Tokens of a padded batch have no expert: all their logits
are -inf, and the rows behind the last used one keep what they held.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: the borders between neighbours
# (a tie goes to the even code) and the step across each.
E2M1_BORDERS = ((0.25, False, 0.5), (0.75, True, 0.5), (1.25, False, 0.5), (1.75, True, 0.5),
                (2.5, False, 1.0), (3.5, True, 1.0), (5.0, False, 2.0))
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step: latency
        dict(name="route_m1_e128_k8", op="route", M=1, E=128, k=8, dtype="bf16", renormalize=True, pad=0),
        # a long prefill batch, fp32 logits, the last tokens padding
        dict(name="route_m16384_e256_k8", op="route", M=16384, E=256, k=8, dtype="fp32", renormalize=True, pad=100),
        # one token to its eight experts
        dict(name="quantize_m1_e128_k8_h2048", op="quantize", M=1, E=128, k=8, H=2048, dtype="bf16", act="none", pad=0),
        # a prefill batch, fanned out
        dict(name="quantize_m8192_e128_k8_h4096", op="quantize", M=8192, E=128, k=8, H=4096, dtype="bf16", act="none",
             pad=0),
        # between the two products of the experts
        dict(name="quantize_m2048_e64_k8_h2048_silu", op="quantize", M=2048, E=64, k=8, H=2048, dtype="bf16",
             act="silu", pad=0),
        # one token: eight weights are read, nothing else matters
        dict(name="linear_m1_e128_k8_n2048_k4096", op="linear", M=1, E=128, k=8, N=2048, K=4096, dtype="bf16",
             bias=False, pad=0),
        # a decode batch: nearly every expert has a few rows, all weights are read
        dict(name="linear_m64_e128_k8_n4096_k2048", op="linear", M=64, E=128, k=8, N=4096, K=2048, dtype="bf16",
             bias=False, pad=0),
        # odd sizes, a bias per expert, a padded batch
        dict(name="linear_m301_e60_k4_n1000_k1088", op="linear", M=301, E=60, k=4, N=1000, K=1088, dtype="fp16",
             bias=True, pad=17),
        # a chunk of a prompt: a few hundred rows per expert
        dict(name="linear_m2048_e64_k8_n4096_k4096", op="linear", M=2048, E=64, k=8, N=4096, K=4096, dtype="bf16",
             bias=False, pad=0),
        # a large prefill batch, the down projection
        dict(name="linear_m8192_e64_k8_n4096_k2048", op="linear", M=8192, E=64, k=8, N=4096, K=2048, dtype="bf16",
             bias=False, pad=0),
        # one token's eight rows
        dict(name="combine_m1_k8_h2048", op="combine", M=1, E=128, k=8, H=2048, dtype="bf16", add=False, pad=0),
        # a prefill batch, a shared expert's output added
        dict(name="combine_m8192_k8_h4096", op="combine", M=8192, E=128, k=8, H=4096, dtype="bf16", add=True, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantize", "linear", "linear", "combine"))
    E, k = _log(rng, 8, 256), rng.randint(1, 8)
    c = dict(op=op, E=E, k=k, dtype=rng.choice(("bf16", "fp16")))
    if op == "route":
        c.update(M=_log(rng, 1, 16384), dtype=rng.choice(("bf16", "fp16", "fp32")), renormalize=rng.random() < 0.5)
    elif op == "quantize":
        act = rng.choice(("none", "silu", "gelu_tanh"))
        H = 64 * _log(rng, 8, 64)
        most = 8192 * 8 * 4096 // (k * H * (1 if act == "none" else 3))
        c.update(M=min(_log(rng, 1, 8192), most), H=H, act=act)
    elif op == "linear":
        E = c["E"] = min(E, 128)
        K, N = 64 * _log(rng, 4, 64), _log(rng, 64, 4096)
        E = c["E"] = max(8, min(E, 128 * 4096 * 2048 // (N * K)))
        c.update(M=min(_log(rng, 1, 8192), 8192 * 8 * 4096 * 2048 // (k * N * K)), N=N, K=K, bias=rng.random() < 0.5)
    else:
        H = 8 * _log(rng, 64, 512)
        c.update(M=min(_log(rng, 1, 8192), 8192 * 8 * 4096 // (k * H)), H=H, add=rng.random() < 0.5)
    c["pad"] = rng.choice((0, c["M"] // 16))
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = DT[case["dtype"]]
    op, M, E, k = (case[n] for n in ("op", "M", "E", "k"))
    R = M * k

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * sd

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")

    s = dict(case)
    # tokens that differ, experts that are more and less popular; a padded batch's last tokens have no expert
    logits = (normal(M, E, sd=1.5) + normal(E, sd=0.7)).to(T)
    if case["pad"]:
        logits[M - case["pad"]:] = -math.inf
    if op == "route":
        s["logits"] = logits
        s["out"] = (ints(M, k), torch.zeros(M, k, device="cuda"), ints(E + 1), ints(M, k))
        return s
    s["experts"], s["weights"], s["offsets"], s["slots"] = _route(logits, k, True, torch.float32)
    s["row_expert"] = _row_expert(s["offsets"], R)
    s["used"] = int(s["offsets"][-1])  # rows that the plain forms look at
    tile_rows = (R // 128 + E) * 128
    if op == "quantize":
        H = case["H"]
        s["x"] = normal(M, H).to(T) if case["act"] == "none" else normal(R, 2 * H).to(T)
        s["scale"] = (200.0 * torch.exp(normal(E, sd=0.2)))
        s["q"] = torch.zeros(R, H // 2, dtype=torch.uint8, device="cuda")
        s["sf"] = torch.zeros(tile_rows, H // 16, dtype=torch.uint8, device="cuda").view(E4M3)
        s["back"] = torch.zeros(R, H, dtype=T if case["act"] == "none" else E4M3, device="cuda")
    elif op == "linear":
        N, K = case["N"], case["K"]
        ga, gw = 400.0 * torch.exp(normal(E, sd=0.2)), 16000.0 * torch.exp(normal(E, sd=0.2))
        row_scale = torch.cat((ga, ga[:1]))[s["row_expert"]]
        v, sf = _nvfp4(normal(R, K).to(T), row_scale)
        s["aq"] = _pack(v)
        s["asf"] = _to_tiles(s, sf, tile_rows)
        s["wq"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        s["wsf"] = torch.empty(E, -(-N // 128) * 128, K // 16, dtype=torch.uint8, device="cuda").view(E4M3)
        for e in range(E):  # one expert's weight at a time: the temporaries are many times its size
            v, sf = _nvfp4(normal(N, K, sd=0.03).to(T), gw[e].expand(N))
            s["wq"][e] = _pack(v)
            s["wsf"][e] = _swizzle(sf)
        s["alpha"] = 1.0 / (ga * gw)
        s["bias_t"] = normal(E, N).to(T) if case["bias"] else None
        s["y"] = torch.zeros(R, N, dtype=T, device="cuda")
        # the plan of the plain products: the experts that have rows, and each row's place in a padded batch of them
        counts = (s["offsets"][1:] - s["offsets"][:-1]).long()
        s["active"] = counts.nonzero()[:, 0]
        s["most"] = int(counts.max())
        place = torch.cumsum((counts > 0).long(), 0) - 1
        e = s["row_expert"][:s["used"]]
        s["at"] = (place[e], torch.arange(s["used"], device="cuda") - s["offsets"].long()[e])
    else:
        H = case["H"]
        s["y"] = normal(R, H).to(T)
        s["add_t"] = normal(M, H).to(T) if case["add"] else None
        s["res"] = torch.zeros(M, H, dtype=T, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _route(logits, k, renormalize, wide):
    """(experts, weights, offsets, slots): the k largest logits of each row, ties to the lowest index."""
    M, E = logits.shape
    v = logits.to(wide)
    top, experts = torch.sort(v, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    chosen = top > -math.inf
    peak = torch.where(chosen[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    w = torch.exp(top - peak)
    total = (w if renormalize else torch.exp(v - peak)).sum(1, keepdim=True)
    w = torch.where(chosen, w / total, torch.zeros_like(w))
    flat = torch.where(chosen, experts, torch.full_like(experts, E)).reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    slots = torch.empty_like(order)
    slots[order] = torch.arange(M * k, device=v.device)
    ends = torch.searchsorted(flat[order], torch.arange(E + 1, device=v.device))
    slots = torch.where(chosen, slots.reshape(M, k), torch.full_like(experts, -1))
    experts = torch.where(chosen, experts, torch.full_like(experts, -1))
    return experts.int(), w.float(), ends.int(), slots.int()


def _row_expert(offsets, R):
    """Expert of each row; E for rows behind the last."""
    return torch.searchsorted(offsets[1:].long(), torch.arange(R, device=offsets.device), right=True)


def _e2m1(v):
    """The E2M1 value nearest to v (ties to the even code, saturating at 6)."""
    a = v.abs()
    r = torch.zeros_like(a)
    for border, tie_up, step in E2M1_BORDERS:
        r = r + step * ((a >= border) if tie_up else (a > border)).to(a.dtype)
    return torch.copysign(r, v)


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(E4M3)


def _nvfp4(x, scale):
    """(E2M1 values (R, K), E4M3 block scales (R, K/16)) of a 16-bit matrix, one global scale per row."""
    R, K = x.shape
    b = x.float().reshape(R, K // 16, 16)
    g = scale.float()[:, None]
    sf = _e4m3(g * (b.abs().amax(-1) / 6.0))
    v = sf.float()
    es = torch.where(v > 0, g / torch.where(v > 0, v, torch.ones_like(v)), torch.zeros_like(v))
    return _e2m1(b * es[..., None]).reshape(R, K), sf


def _swizzle(sf):
    """(M, Kb) block scales in the 128x4 layout: (round_up(M, 128), Kb), padding 0."""
    M, Kb = sf.shape
    Mp = -(-M // 128) * 128
    p = torch.zeros(Mp, Kb, dtype=torch.uint8, device=sf.device)
    p[:M] = sf.view(torch.uint8)
    return p.reshape(Mp // 128, 4, 32, Kb // 4, 4).permute(0, 3, 2, 1, 4).reshape(Mp, Kb).view(E4M3)


def _unswizzle(sw):
    Mp, Kb = sw.shape
    p = sw.contiguous().view(torch.uint8).reshape(Mp // 128, Kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return p.reshape(Mp, Kb).view(E4M3)


def _tile_row(s):
    """Row of the unswizzled scale tiles of each used row."""
    e = s["row_expert"][:s["used"]]
    o = s["offsets"].long()[e]
    return (o // 128 + e) * 128 + torch.arange(s["used"], device=e.device) - o


def _to_tiles(s, sf, tile_rows):
    """(R, Kb) block scales in the tiles of the expert order, padding 0."""
    p = torch.zeros(tile_rows, sf.shape[1], dtype=torch.uint8, device=sf.device)
    p[_tile_row(s)] = sf[:s["used"]].view(torch.uint8)
    return _swizzle(p.view(E4M3))


def _pack(values):
    a = values.abs()
    mag = torch.where(a <= 2.0, a * 2.0, torch.where(a == 6.0, a + 1.0, a + 2.0)).to(torch.uint8)
    code = mag | (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(q, sf):
    """code * block scale (plain order), exact in fp32."""
    lut = torch.tensor(E2M1_VALUES, dtype=torch.float32, device=q.device)
    v = lut[torch.stack((q & 15, q >> 4), -1).to(torch.int32)].reshape(*sf.shape, 16)
    return (v * sf.float()[..., None]).reshape(*q.shape[:-1], 2 * q.shape[-1])


def _act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    return g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain(s):
    op, T, E = s["op"], DT[s["dtype"]], s["E"]
    if op == "route":
        return _route(s["logits"], s["k"], s["renormalize"], torch.float32)
    R = s["M"] * s["k"]
    if op == "quantize":
        H, e = s["H"], s["row_expert"]
        if s["act"] == "none":
            token = torch.zeros(R + 1, dtype=torch.long, device="cuda")
            to = s["slots"].reshape(-1).long()
            token[torch.where(to < 0, torch.full_like(to, R), to)] = torch.arange(R, device="cuda") // s["k"]
            y = s["x"][token[:R]]
        else:
            x = s["x"].float()
            y = (_act(x[:, :H], s["act"]) * x[:, H:]).to(T)
        g = torch.cat((s["scale"], s["scale"][:1]))[e]
        v, sf = _nvfp4(y, g)
        back = v.reshape(R, H // 16, 16) * (sf.float() / g[:, None])[..., None]
        back = torch.where((e < E)[:, None], back.reshape(R, H), torch.zeros_like(v))
        tiles = _to_tiles(s, sf, s["sf"].shape[0])
        return (back.to(T) if s["act"] == "none" else _e4m3(back)), tiles
    if op == "linear":
        used, K = s["used"], s["K"]
        rows = _unswizzle(s["asf"])[_tile_row(s)]
        a = torch.zeros(s["active"].numel(), s["most"], K, device="cuda")
        a[s["at"]] = _values(s["aq"][:used], rows)
        wsf = s["wsf"].view(torch.uint8)[s["active"]].view(E4M3)
        n = wsf.shape[1]
        w = _values(s["wq"][s["active"]], _unswizzle(wsf.reshape(-1, K // 16)).reshape(-1, n, K // 16)[:, :s["N"]])
        y = torch.bmm(a, w.transpose(1, 2)) * s["alpha"][s["active"]][:, None, None]
        if s["bias_t"] is not None:
            y = y + s["bias_t"].float()[s["active"]][:, None]
        out = torch.zeros(R, s["N"], dtype=T, device="cuda")
        out[:used] = y.to(T)[s["at"]]
        return (out,)
    to, w = s["slots"].long(), s["weights"]
    rows = s["y"][to.clamp(min=0)].float()
    out = (torch.where((to >= 0)[..., None], rows, torch.zeros_like(rows)) * w[..., None]).sum(1)
    if s["add_t"] is not None:
        out = out + s["add_t"].float()
    return (out.to(T),)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    if own:
        import nvfp4_quant_gemma_gb300 as gnq
        op = s["op"]
        if op == "route":
            return gnq.expert_route(s["logits"], s["k"], renormalize=s["renormalize"], out=s["out"])
        if op == "quantize":
            fan = s["act"] == "none"
            q, sf = gnq.expert_quantize(s["x"], s["offsets"], s["scale"], slots=s["slots"] if fan else None,
                                        experts=s["experts"] if fan else None, act=None if fan else s["act"],
                                        out=(s["q"], s["sf"]))
            return gnq.expert_dequantize(q, sf, s["offsets"], s["scale"], out=s["back"]), sf
        if op == "linear":
            return gnq.nvfp4_expert_linear(s["aq"], s["asf"], s["wq"], s["wsf"], s["alpha"], s["offsets"],
                                           bias=s["bias_t"], out=s["y"]),
        return gnq.expert_combine(s["y"], s["slots"], s["weights"], add=s["add_t"], out=s["res"]),
    return _plain(s)


def work(case):
    op, E, k = case["op"], case["E"], case["k"]
    M = case["M"] - case["pad"]
    R = M * k
    if op == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=case["M"] * E * size + 12 * case["M"] * k + 4 * E, flops=case["M"] * E * (k + 8))
    if op == "quantize":
        n = R * case["H"]
        nvfp4 = n * 9 / 16  # codes and block scales: written by one call, read by the next
        if case["act"] == "none":
            return dict(bytes=2 * M * case["H"] + 4 * R + 2 * nvfp4 + 2 * n, flops=8 * n)
        return dict(bytes=4 * n + 2 * nvfp4 + n, flops=20 * n)
    if op == "linear":
        # experts that have rows, as if each token's k were drawn evenly
        N, K, active = case["N"], case["K"], E * (1.0 - (1.0 - min(1.0, k / E)) ** M)
        return dict(bytes=(active * N + R) * K * 9 / 16 + 2 * R * N + (2 * active * N if case["bias"] else 0),
                    flops=2 * R * N * K)
    H = case["H"]
    return dict(bytes=2 * R * H + 8 * R + 2 * case["M"] * H * (2 if case["add"] else 1), flops=2 * R * H)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    """Outputs from the definitions in fp64.  Choices by repeated maxima and
    counting, 4-bit and 8-bit steps by a search among all code values, scales
    placed by the layout's byte formula, products one expert at a time: unlike
    the plain forms."""
    s = prepare(case, seed)
    f64, T = torch.float64, DT[case["dtype"]]
    op, M, E, k = (case[n] for n in ("op", "M", "E", "k"))
    R = M * k
    if op == "route":
        left = s["logits"].to(f64)
        mass = torch.exp(left - left.amax(1, keepdim=True))
        mass = torch.where(torch.isnan(mass), torch.zeros_like(mass), mass)
        index = torch.arange(E, device="cuda")
        experts = torch.full((M, k), -1, dtype=torch.int32, device="cuda")
        weights = torch.zeros(M, k, dtype=f64, device="cuda")
        for j in range(k):
            best = left.amax(1, keepdim=True)
            pick = torch.where(left == best, index, E).amin(1)
            live = best[:, 0] > -math.inf
            experts[:, j] = torch.where(live, pick, -torch.ones_like(pick)).int()
            weights[:, j] = torch.where(live, mass.gather(1, pick[:, None])[:, 0], torch.zeros_like(weights[:, j]))
            left = left.scatter(1, pick[:, None], -math.inf)
        total = weights.sum(1) if case["renormalize"] else mass.sum(1)
        weights = weights / torch.where(total > 0, total, torch.ones_like(total))[:, None]
        one = torch.zeros(M, E + 1, dtype=torch.int64, device="cuda")
        one.scatter_(1, torch.where(experts < 0, E, experts).long(), 1)
        before = one.cumsum(0) - one
        ends = one.sum(0)[:E].cumsum(0)
        offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
        at = experts.clamp(min=0).long()
        slots = torch.where(experts < 0, torch.full_like(at, -1), offsets[at] + before.gather(1, at))
        return experts, weights, offsets.int(), slots.int()

    bounds = s["offsets"].tolist()
    e2 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=f64, device="cuda")
    e4 = torch.arange(127, dtype=torch.uint8, device="cuda").view(E4M3).to(f64)  # 0 .. 448, ascending

    def nearest(v, values):
        """Index of the value nearest to |v|: the lower neighbour, or the upper one where it is nearer or a tie's even code."""
        a = v.abs().clamp(max=float(values[-1]))
        lo = (torch.searchsorted(values, a, right=True) - 1).clamp(0, len(values) - 2)
        down, up = a - values[lo], values[lo + 1] - a
        return lo + ((up < down) | ((up == down) & (lo % 2 == 1))).to(lo.dtype)

    def places(rows, tile, Kb):
        """Byte of each block scale of `rows` rows whose first tile is `tile`."""
        m = torch.arange(rows, device="cuda")[:, None]
        b = torch.arange(Kb, device="cuda")[None, :]
        return ((tile + m // 128) * (Kb // 4) + b // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + b % 4

    if op == "quantize":
        H = case["H"]
        back = torch.zeros_like(s["back"])
        codes = torch.zeros(s["sf"].numel(), dtype=torch.uint8, device="cuda")
        source = torch.zeros(R, dtype=torch.long, device="cuda")
        t, j = (s["slots"] >= 0).nonzero(as_tuple=True)
        source[s["slots"][t, j].long()] = t
        for e in range(E):
            a, z = bounds[e], bounds[e + 1]
            if a == z:
                continue
            if case["act"] == "none":
                y = s["x"][source[a:z]]
            else:
                p, u = s["x"][a:z].to(f64).split(H, 1)
                if case["act"] == "silu":
                    p = p * torch.sigmoid(p)
                else:
                    p = 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p.pow(3))))
                y = (p * u).to(T)
            g = float(s["scale"][e])
            b = y.to(f64).unflatten(1, (H // 16, 16))
            c = nearest(g * b.abs().amax(2) / 6.0, e4)
            v = e4[c]
            x = b * (g / v)[..., None]
            x = torch.where(v[..., None] == 0, torch.zeros_like(x), x)
            x = (torch.copysign(e2[nearest(x, e2)], x) * v[..., None] / g).flatten(1)
            if case["act"] != "none":
                x = torch.copysign(e4[nearest(x, e4)], x)
            back[a:z] = x.to(back.dtype)
            codes[places(z - a, a // 128 + e, H // 16).reshape(-1)] = c.to(torch.uint8).reshape(-1)
        return back, codes.reshape(-1, H // 16).view(E4M3)
    if op == "linear":
        N, K = case["N"], case["K"]
        sign = torch.cat((e2, -e2))

        def matrix(q, sf, tile):
            v = torch.empty(q.shape[0], K, dtype=f64, device="cuda")
            v[:, 0::2] = sign[(q % 16).long()]
            v[:, 1::2] = sign[(q // 16).long()]
            return v * sf.reshape(-1)[places(q.shape[0], tile, K // 16)].to(f64).repeat_interleave(16, 1)

        y = torch.zeros_like(s["y"])
        for e in range(E):
            a, z = bounds[e], bounds[e + 1]
            if a == z:
                continue
            p = torch.mm(matrix(s["aq"][a:z], s["asf"], a // 128 + e), matrix(s["wq"][e], s["wsf"][e], 0).t())
            p = p * float(s["alpha"][e])
            if case["bias"]:
                p = p + s["bias_t"][e].to(f64)
            y[a:z] = p.to(T)
        return (y,)
    out = s["add_t"].to(f64) if case["add"] else torch.zeros(M, case["H"], dtype=f64, device="cuda")
    for j in range(k):
        to = s["slots"][:, j].long()
        live = to >= 0
        out[live] += s["y"][to[live]].to(f64) * s["weights"][live, j].to(f64)[:, None]
    return (out.to(T),)
