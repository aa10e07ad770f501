"""Measured cases of the operators beside the quantized linear layer.

Three operators, each bf16 in and out:

  group_norm  group norm with an activation over channels-last activations
              [B, S, C] (S pixels of C channels), the producer of a 1x1
              convolution's input:
                y = act((x - mean) / sqrt(var + eps) * gamma_c + beta_c)
  dense       the 16-bit matrix product with bias, activation, gate and
              residual in its epilogue (layers that stay in 16 bits):
                Y = R + g * act(X W^T + b)
  linear      the quantized layer's integer product with the same epilogue:
                Y = R + g * act(s_x s_w (A B^T) + b + m colsum)

The gate g has one row per `gate_rows` rows of Y (a sample's modulation).
`own = False` computes the plain forms with elementary torch operations in 32
bits (64 where an integer sum needs it), rounded once at the end; `own = True`
makes the library's calls.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------- cases
def _gn(name, B, S, C, G, act):
    return {"name": name, "op": "group_norm", "B": B, "S": S, "C": C, "G": G, "act": act}


def _dense(name, T, K, N, act, bias=True, residual=False, gate_rows=0):
    return {"name": name, "op": "dense", "T": T, "K": K, "N": N, "act": act, "bias": bias,
            "residual": residual, "gate_rows": gate_rows}


def _linear(name, T, K, N, a_bits, w_bits, act, per_token=True, mean=True, packed=False,
            residual=False, gate_rows=0):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "a_bits": a_bits,
            "w_bits": w_bits, "act": act, "per_token": per_token, "mean": mean,
            "packed": packed, "residual": residual, "gate_rows": gate_rows}


def listed():
    return [
        # one latent image of 64 x 64 pixels before a 1x1 convolution: latency
        _gn("gn_one_latent", 1, 4096, 320, 32, "silu"),
        # the 65536 pixels of the 1x1 convolution configuration, as 16 images
        _gn("gn_batch_latents", 16, 4096, 320, 32, "silu"),
        # one image of 512 x 512 pixels in a decoder's last stage
        _gn("gn_full_image", 1, 262144, 128, 32, "silu"),
        # odd numbers of pixels and channels per group, no activation
        _gn("gn_odd", 3, 5041, 182, 26, "none"),
        # the timestep embedding's first layer, one row per sample: latency
        _dense("dense_timestep", 2, 256, 1152, "silu"),
        # the modulation vectors of a block (6 x 1152) for a batch of 4
        _dense("dense_modulation", 4, 1152, 6912, "none"),
        # an MLP's second layer kept in 16 bits: gated and added to the stream,
        # in images of 1000 tokens (no multiple of a tile)
        _dense("dense_fc2_odd", 7000, 4608, 1152, "none", residual=True, gate_rows=1000),
        # the largest product
        _dense("dense_large", 16384, 4096, 8192, "gelu_tanh"),
        # one token through the qkv-sized quantized layer
        _linear("linear_one_token", 1, 1152, 3456, 4, 4, "none"),
        # an MLP's first layer, 4-bit codes, GELU
        _linear("linear_fc1", 8192, 1152, 4608, 4, 4, "gelu_tanh"),
        # an MLP's second layer, 3-bit activations, gated and added
        _linear("linear_fc2", 8192, 4608, 1152, 3, 4, "none", residual=True, gate_rows=4096),
        # the 1x1 convolution with 8-bit codes, per-tensor scale, added to its input
        _linear("linear_conv1x1", 65536, 320, 320, 8, 8, "silu", per_token=False, mean=False,
                residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("group_norm", "dense", "linear"))
    if op == "group_norm":
        G = rng.choice((1, 7, 8, 16, 32))
        C = G * _log_int(rng, 2, 40)
        B = _log_int(rng, 1, 16)
        S = _log_int(rng, 1, max(2, min(262144, 33_000_000 // (B * C))))
        c = _gn("", B, S, C, G, rng.choice(ACTS))
    elif op == "dense":
        K = 8 * _log_int(rng, 8, 576)
        N = 8 * _log_int(rng, 2, 1024)
        T = _log_int(rng, 1, min(16384, 550_000_000_000 // (K * N)))
        c = _dense("", T, K, N, rng.choice(ACTS), rng.random() < 0.8, rng.random() < 0.5,
                   rng.choice((0, 0, 1, 100, 1024)))
    else:
        a_bits = rng.choice((3, 4, 8))
        w_bits = rng.choice((4, 8))
        packed = a_bits < 8 and rng.random() < 0.25
        K = (32 if packed else 16) * _log_int(rng, 4, 288 if packed else 576)
        N = 16 * _log_int(rng, 1, 512)
        T = _log_int(rng, 1, min(65536, 250_000_000_000 // (K * N)))
        per_token = rng.random() < 0.7
        c = _linear("", T, K, N, a_bits, w_bits, rng.choice(ACTS), per_token,
                    per_token and rng.random() < 0.7, packed, rng.random() < 0.5,
                    rng.choice((0, 0, 1, 100, 1024)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "group_norm":
        B, S, C = case["B"], case["S"], case["C"]
        # channels of different spread and offset, as a convolution leaves them
        x = randn(B, S, C)
        x *= torch.exp(0.7 * randn(1, 1, C))
        x += 1.5 * randn(B, 1, C)
        st["x"] = x.to(torch.bfloat16)
        st["gamma"] = (1.0 + 0.3 * randn(C)).to(torch.bfloat16)
        st["beta"] = (0.3 * randn(C)).to(torch.bfloat16)
        return st
    T, K, N = case["T"], case["K"], case["N"]
    if case["op"] == "dense":
        st["x"] = randn(T, K).to(torch.bfloat16)
        # weights that keep the outputs at the inputs' scale
        st["w"] = (randn(N, K) * K ** -0.5).to(torch.bfloat16)
        st["bias"] = (0.3 * randn(N)).to(torch.bfloat16) if case["bias"] else None
    else:
        qa, qw = 2 ** (case["a_bits"] - 1) - 1, 2 ** (case["w_bits"] - 1) - 1
        # codes as the quantizers leave them: a bell whose largest reaches q
        codes = (randn(T, K) * (qa / 3.5)).round_().clamp_(-qa, qa).to(torch.int8)
        if case["packed"]:  # two 4-bit codes a byte, the even element in the low nibble
            lo, hi = codes[:, 0::2].to(torch.int16), codes[:, 1::2].to(torch.int16)
            st["a_codes"] = ((lo & 15) | ((hi & 15) << 4)).to(torch.uint8)
        else:
            st["a_codes"] = codes
        st["w_codes"] = (randn(N, K) * (qw / 3.5)).round_().clamp_(-qw, qw).to(torch.int8)
        # scales that bring the sums to about one
        rows = T if case["per_token"] else 1
        st["a_scale"] = torch.exp(0.3 * randn(rows)) * (3.5 / qa)
        st["w_scale"] = torch.exp(0.1 * randn(N)) * (3.5 / qw) * K ** -0.5
        st["a_mean"] = randn(T) * 0.1 if case["mean"] else None
        st["colsum"] = randn(N)
        st["bias"] = 0.3 * randn(N)
    st["residual"] = randn(T, N).to(torch.bfloat16) if case["residual"] else None
    gr = case["gate_rows"]
    st["gate"] = (0.5 * randn((T + gr - 1) // gr, N)).to(torch.bfloat16) if gr else None
    return st


# -------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _finish(z, st):
    """R + g * act(z), rounded once."""
    case = st["case"]
    y = _act(z, case["act"])
    if st["gate"] is not None:
        y = y * st["gate"].float().repeat_interleave(case["gate_rows"], dim=0)[: case["T"]]
    if st["residual"] is not None:
        y = st["residual"].float() + y
    return y.to(torch.bfloat16)


def _codes(st):
    if not st["case"]["packed"]:
        return st["a_codes"]
    b = st["a_codes"].to(torch.int16)
    lo, hi = b & 15, b >> 4
    pair = torch.stack((lo - 16 * (lo > 7), hi - 16 * (hi > 7)), dim=-1)
    return pair.reshape(st["case"]["T"], st["case"]["K"])


def _plain(st):
    case = st["case"]
    if case["op"] == "group_norm":
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        x = st["x"].float().view(B, S, G, C // G)
        mean = x.mean(dim=(1, 3), keepdim=True)
        d = x - mean
        var = (d * d).mean(dim=(1, 3), keepdim=True)
        y = (d / torch.sqrt(var + 1e-5)).view(B, S, C)
        return _act(y * st["gamma"].float() + st["beta"].float(), case["act"]).to(torch.bfloat16)
    if case["op"] == "dense":
        z = st["x"].float() @ st["w"].float().t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        return _finish(z, st)
    # sums of code products are whole numbers: exact in 32 bits below 2^24
    bound = 2 ** (case["a_bits"] + case["w_bits"] - 2) * case["K"]
    t = torch.float32 if bound < 2 ** 24 else torch.float64
    acc = (_codes(st).to(t) @ st["w_codes"].to(t).t()).float()
    z = acc * (st["a_scale"][:, None] * st["w_scale"]) + st["bias"]
    if st["a_mean"] is not None:
        z = z + st["a_mean"][:, None] * st["colsum"]
    return _finish(z, st)


# --------------------------------------------------------- the library's calls
def _own(st):
    import hadamard_rotated_bit_token_b200 as hq
    case = st["case"]
    if case["op"] == "group_norm":
        norm = st.get("norm")
        if norm is None:  # the layer that a program keeps
            norm = st["norm"] = hq.GroupNorm(case["C"], case["G"], st["gamma"], st["beta"],
                                             eps=1e-5, act=ACTS.index(case["act"]))
        return norm(st["x"])
    act = ACTS.index(case["act"])
    if case["op"] == "dense":
        layer = st.get("layer")
        if layer is None:
            layer = st["layer"] = hq.DenseLinear(st["w"], st["bias"], act=act)
        return layer(st["x"], residual=st["residual"], gate=st["gate"],
                     gate_rows=case["gate_rows"])
    desc = st.get("desc")
    if desc is None:
        desc = st["desc"] = hq.LayerDesc(
            case["K"], case["N"], 16, a_bits=case["a_bits"], w_bits=case["w_bits"],
            act_gran=hq.HQ_PER_TOKEN if case["per_token"] else hq.HQ_PER_TENSOR_DYNAMIC,
            centering=hq.HQ_CENTER_TOKEN_MEAN if case["mean"] else hq.HQ_CENTER_NONE,
            code_format=hq.HQ_CODES_I4_PACKED if case["packed"] else hq.HQ_CODES_I8)
    Y = torch.empty((case["T"], case["N"]), dtype=torch.bfloat16, device="cuda")
    ep = hq.Epilogue(act, residual=st["residual"], gate=st["gate"], gate_rows=case["gate_rows"])
    hq.hq_linear_ep(desc, st["a_codes"], st["a_scale"], st["a_mean"], st["w_codes"],
                    st["w_scale"], st["colsum"], st["bias"], ep, Y)
    return Y


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "group_norm":
        n = case["B"] * case["S"] * case["C"]
        return {"bytes": 4 * n + 4 * case["C"], "flops": 10 * n}
    T, K, N = case["T"], case["K"], case["N"]
    gr = case["gate_rows"]
    b = 2 * T * N * (2 if case["residual"] else 1) + (2 * N * ((T + gr - 1) // gr) if gr else 0)
    if case["op"] == "dense":
        b += 2 * (T * K + N * K) + (2 * N if case["bias"] else 0)
    else:
        b += (T * K // 2 if case["packed"] else T * K) + N * K + 8 * N
        b += 4 * (T if case["per_token"] else 1) + (4 * T + 4 * N if case["mean"] else 0)
    return {"bytes": b, "flops": 2 * T * K * N}


# ------------------------------------------------------- definitions, 64 bits
def _phi(z):
    """The normal distribution function."""
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * _phi(z)
    # 0.5 (1 + tanh u) = sigmoid(2 u)
    return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


def exact(case, seed):
    st = prepare(case, seed)
    act = case["act"]
    if case["op"] == "group_norm":
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        out = []
        for xb in st["x"]:  # one image at a time: [S, C] -> groups as rows
            x = xb.double().t().reshape(G, -1)
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            n = ((x - mean) * torch.rsqrt(var + 1e-5)).view(C, S)
            n = n * st["gamma"].double()[:, None] + st["beta"].double()[:, None]
            out.append(_exact_act(n, act).t())
        return torch.stack(out)
    T, K, N = case["T"], case["K"], case["N"]
    step = max(1, 2 ** 28 // (K + 4 * N))  # rows at a time
    out = []
    w = (st["w"] if case["op"] == "dense" else st["w_codes"]).double()
    codes = None if case["op"] == "dense" else _unpacked(st)
    for i in range(0, T, step):
        j = min(T, i + step)
        if case["op"] == "dense":
            z = torch.einsum("tk,nk->tn", st["x"][i:j].double(), w)
        else:
            z = torch.einsum("tk,nk->tn", codes[i:j].double(), w)
            sx = st["a_scale"].double()
            z = z * (sx[i:j] if case["per_token"] else sx)[:, None] * st["w_scale"].double()
            if case["mean"]:
                z = z + torch.outer(st["a_mean"][i:j].double(), st["colsum"].double())
        if st["bias"] is not None:
            z = z + st["bias"].double()
        y = _exact_act(z, act)
        if st["gate"] is not None:
            rows = torch.arange(i, j, device="cuda") // case["gate_rows"]
            y = y * st["gate"][rows].double()
        if st["residual"] is not None:
            y = y + st["residual"][i:j].double()
        out.append(y)
    return torch.cat(out)


def _unpacked(st):
    """Activation codes as whole numbers, from packed nibbles where they are."""
    if not st["case"]["packed"]:
        return st["a_codes"]
    b = st["a_codes"].view(torch.int8)
    lo = ((b << 4) >> 4) if b.dtype == torch.int8 else b
    hi = b >> 4
    return torch.stack((lo, hi), dim=2).flatten(1)
