"""The per-GPU wo_b step: the four library calls of one row-parallel layer's
local work, on preallocated device buffers.

  1. bsgemm_fp8   C = A x B^T as P destination-major bands of M/P rows
  2. band_reduce  band 0 of C (this GPU's own band) + P-1 partial bands that
                  stand in for the bands the other ranks would send
  3. rowq_e4m3    the reduced band -> e4m3 + per-row scale (the fp8 wire),
                  written into rows [0, M/P) of the gathered wire buffer
  4. rowdq_e4m3   the gathered wire buffer [M, N] (own rows + P-1 stand-in
                  quantized bands) -> bf16

("MORI GEMM + All-Reduce Benchmark", "Where the time goes": gemm, reduce,
quantize, dequantize; the scatter and gather transfers between them are
collectives and are not part of a single-GPU step.)  With ``fused=True``
steps 2 and 3 are one call, band_rowq_e4m3, which writes the same codes and
scales without the reduced bf16 band in memory (the pages' "Negative
results" fusion).  Buffers are allocated once in the constructor; ``step()``
only enqueues the calls on the current stream, so it can be timed or
captured.

``WoBServeStep`` is the same layer as a serving stack runs it: a bf16 input, low-rank
adapters of many requests beside the weight, and the gathered wire taken
straight into the residual stream and the next projection's fp8 operand.

``FFNServeStep`` is the feed-forward block that takes over there: the dense or shared
part as two products with their epilogues, and the routed experts of a few tokens.
"""
import torch

from . import (actq_e4m3, band_reduce, band_rowq_e4m3, bsgemm_fp8, bsgemm_fp8_act, bsgemm_fp8_lora, lora_expand,
               lora_plan, lora_shrink, moe_fp8, moe_fp8_workspace, moe_route, resnorm, rowdq_e4m3, rowq_e4m3)


class WoBStep:
    def __init__(self, A, a_scale, B, b_scale, partials, wire_q, wire_s, bands, fused=False):
        """A/a_scale/B/b_scale: GEMM operands on the device.
        partials: list of bands-1 bf16 [M/bands, N] tensors (the other ranks' bands).
        wire_q/wire_s: uint8 [M, N] and fp32 [M] gathered wire; rows [0, M/bands)
        are overwritten by this GPU's quantized band each step.
        fused: reduce and quantize in one call (band_rowq_e4m3)."""
        M, K = A.shape
        N = B.shape[0]
        if M % bands:
            raise ValueError("M must be a multiple of bands")
        if len(partials) != bands - 1:
            raise ValueError("need bands-1 partial bands")
        self.M, self.N, self.K, self.bands = M, N, K, bands
        self.band_rows = M // bands
        self.A, self.a_scale, self.B, self.b_scale = A, a_scale, B, b_scale
        dev = A.device
        self.C = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        self.partials = list(partials)
        self.fused = fused
        self.PHASES = self.PHASES_FUSED if fused else self.PHASES_SPLIT
        self.reduced = None if fused else torch.empty((self.band_rows, N), dtype=torch.bfloat16, device=dev)
        self.wire_q, self.wire_s = wire_q, wire_s
        self.own_q = wire_q[: self.band_rows]
        self.own_s = wire_s[: self.band_rows]
        self.out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)

    def gemm(self):
        bsgemm_fp8(self.A, self.a_scale, self.B, self.b_scale, self.C.view(-1), bands=self.bands)

    def reduce(self):
        band_reduce([self.C[: self.band_rows]] + self.partials, self.reduced)

    def quantize(self):
        rowq_e4m3(self.reduced, self.own_q, self.own_s)

    def reduce_quantize(self):
        band_rowq_e4m3([self.C[: self.band_rows]] + self.partials, self.own_q, self.own_s)

    def dequantize(self):
        rowdq_e4m3(self.wire_q, self.wire_s, self.out)

    PHASES_SPLIT = ("gemm", "reduce", "quantize", "dequantize")
    PHASES_FUSED = ("gemm", "reduce_quantize", "dequantize")

    def step(self):
        for ph in self.PHASES:
            getattr(self, ph)()


class WoBServeStep:
    """One rank's part of the layer between two collectives' worth of data:

      1. actq_e4m3        x -> the GEMM's fp8 operand
      2. lora_plan, lora_shrink   H = x A[a]^T for each row's adapter (x and A hold
                          this rank's part of K, so H and the adapters' share of
                          the output are partial sums like the GEMM's)
      3. bsgemm_fp8_lora  the partial output, adapters included, as row bands; with
                          fused=False bsgemm_fp8 and lora_expand in place, which a
                          long batch wants whose rows mix many adapters (bsgemm.h
                          has the measurements), at one more rounding of C to bf16
      4. band_rowq_e4m3   this rank's band and the other ranks' -> wire rows
      5. resnorm          the gathered wire -> norm, gate, residual, norm, and the
                          next projection's operand (q, q_scale)

    The plan depends on ids only; a stack of layers makes it once per batch.
    ids, x, resid and the wire's other rows may be refilled between steps: every
    buffer is allocated here and step() only enqueues, so it can be captured.
    """

    PHASES = ("quantize", "plan", "shrink", "gemm", "reduce_quantize", "norm")

    def __init__(self, x, B, b_scale, partials, wire_q, wire_s, bands, resid, ids, lora_A, lora_B, lora_scale=None,
                 post_w=None, gate=None, pre_w=None, alpha=1.0, beta=1.0, eps=1e-6, quant=128, fused=True):
        """x bf16 [M, K]; B, b_scale: the weight; partials, wire_q, wire_s, bands as
        for WoBStep; resid bf16 or fp32 [M, N]; ids int32 [M]; lora_A [L, R, K] and
        lora_B [L, N, R] bf16; the rest as for resnorm."""
        M, K = x.shape
        N = B.shape[0]
        if M % bands:
            raise ValueError("M must be a multiple of bands")
        if len(partials) != bands - 1:
            raise ValueError("need bands-1 partial bands")
        L, R = lora_A.shape[:2]
        dev = x.device

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.x, self.B, self.b_scale, self.bands, self.fused = x, B, b_scale, bands, fused
        self.ids, self.lora_A, self.lora_B, self.lora_scale = ids, lora_A, lora_B, lora_scale
        self.resid, self.wire_q, self.wire_s = resid, wire_q, wire_s
        self.partials = list(partials)
        self.norm_args = dict(post_w=post_w, gate=gate, pre_w=pre_w, alpha=alpha, beta=beta, eps=eps, quant=quant)
        self.A, self.a_scale = new((M, K), torch.uint8), new((M, K // 128), torch.float32)
        self.lora_plan, self.H = new((L + 2 + M,), torch.int32), new((M, R), torch.float32)
        self.C = new((M, N), torch.bfloat16)
        rows = M // bands
        self.own_band, self.own_q, self.own_s = self.C[:rows], wire_q[:rows], wire_s[:rows]
        self.resid_out = torch.empty_like(resid)
        self.z = None if quant else new((M, N), torch.bfloat16)
        self.q = new((M, N), torch.uint8) if quant else None
        self.q_scale = new((M, N // quant), torch.float32 if quant == 128 else torch.uint8) if quant else None

    def quantize(self):
        actq_e4m3(self.x, self.A, self.a_scale)

    def plan(self):
        lora_plan(self.ids, self.lora_A.shape[0], self.lora_plan)

    def shrink(self):
        lora_shrink(self.x, self.lora_A, self.lora_plan, self.H)

    def gemm(self):
        C = self.C.view(-1)
        if self.fused:
            bsgemm_fp8_lora(self.A, self.a_scale, self.B, self.b_scale, self.H, self.lora_B, self.ids, self.lora_scale,
                            C, bands=self.bands)
        else:
            bsgemm_fp8(self.A, self.a_scale, self.B, self.b_scale, C, bands=self.bands)
            lora_expand(self.H, self.lora_B, self.lora_plan, C, C, self.lora_scale, bands=self.bands)

    def reduce_quantize(self):
        band_rowq_e4m3([self.own_band] + self.partials, self.own_q, self.own_s)

    def norm(self):
        resnorm(self.wire_q, self.resid, y_scale=self.wire_s, resid_out=self.resid_out, z=self.z, q=self.q,
                q_scale=self.q_scale, **self.norm_args)

    def step(self):
        for ph in self.PHASES:
            getattr(self, ph)()


class FFNServeStep:
    """One feed-forward block on resnorm's outputs, z (bf16) and q with q_scale (fp32 per
    1x128 block):

      1. up          h = act(q W1^T) * (q W3^T), the dense part (a layer's only expert or the
                     one that all tokens share): bsgemm_fp8_act, gated
      2. quantize    h -> the second product's fp8 operand (actq_e4m3)
      3. down        out = h W2^T (bsgemm_fp8_act)
      4. logits      z router^T in fp32: lora_shrink with the router as every row's adapter
      5. route       each token's experts and weights (moe_route)
      6. experts     out += the experts' weighted outputs (moe_fp8)

    Without a dense part 4 to 6 alone, which need no q; without a router 1 to 3 alone, for any
    number of rows, which need no z.  Experts: up to 128 rows.  The next resnorm takes out as
    its y.  z, q and q_scale may be refilled between steps: every buffer is allocated here
    and step() only enqueues, so it can be captured.
    The router's plan is made here, once, on the current stream.
    """

    DENSE, ROUTED = ("up", "quantize", "down"), ("logits", "route", "experts")

    def __init__(self, z=None, q=None, q_scale=None, dense=None, router=None, experts=None, topk=1, act="silu",
                 bias=None, **route):
        """z bf16 [M, D]; q uint8 [M, D], q_scale fp32 [M, D/128]; dense: (B13, s13, B2, s2), the weight
        [2I, D], W1's rows first, and [D, I] with their scales, or None; router: bf16 [E, D], E a
        multiple of 8 up to 256, with experts: (W13, s13, W2, s2) as for moe_fp8, or None;
        topk, bias and route (score, groups, ...): as for moe_route."""
        if (router is None) != (experts is None):
            raise ValueError("router and experts go together")
        if dense is None and experts is None:
            raise ValueError("need a dense part, experts or both")
        if dense is not None and (q is None or q_scale is None):
            raise ValueError("the dense part needs q and q_scale")
        if experts is not None and z is None:
            raise ValueError("the experts need z")
        M, D = (q if z is None else z).shape
        dev = (q if z is None else z).device
        if dense is not None:   # what the calls cannot see: each would write a part of its buffer alone
            I = dense[2].shape[1]
            for name, t, shape in (("q", q, (M, D)), ("dense B13", dense[0], (2 * I, D)), ("dense B2", dense[2], (D, I))):
                if tuple(t.shape) != shape:
                    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.z, self.q, self.q_scale, self.act, self.topk = z, q, q_scale, act, topk
        self.dense, self.router, self.expert_weights, self.bias, self.route_args = dense, router, experts, bias, route
        self.out = new((M, D), torch.bfloat16)
        self.PHASES = (self.DENSE if dense is not None else ()) + (self.ROUTED if experts is not None else ())
        if dense is not None:
            self.h = new((M, I), torch.bfloat16)
            self.hq, self.h_scale = new((M, I), torch.uint8), new((M, I // 128), torch.float32)
        if experts is not None:
            E, rows = experts[0].shape[:2]
            if router.shape[0] != E:
                raise ValueError(f"the router has {router.shape[0]} experts, the weights {E}")
            self.router = router.view(1, E, D)
            self.plan = lora_plan(torch.zeros(M, dtype=torch.int32, device=dev), 1)
            self.router_logits = new((M, E), torch.float32)
            self.ids, self.weights = new((M, topk), torch.int32), new((M, topk), torch.float32)
            self.ws = new(moe_fp8_workspace(M, topk, E, rows // 2), torch.uint8)

    def up(self):
        bsgemm_fp8_act(self.q, self.q_scale, *self.dense[:2], act=self.act, gated=True, C=self.h)

    def quantize(self):
        actq_e4m3(self.h, self.hq, self.h_scale)

    def down(self):
        bsgemm_fp8_act(self.hq, self.h_scale, *self.dense[2:], C=self.out)

    def logits(self):
        lora_shrink(self.z, self.router, self.plan, self.router_logits)

    def route(self):
        moe_route(self.router_logits, self.topk, bias=self.bias, ids=self.ids, weights=self.weights, **self.route_args)

    def experts(self):
        moe_fp8(self.z, self.ids, self.weights, *self.expert_weights, base=None if self.dense is None else self.out,
                act=self.act, out=self.out, ws=self.ws)

    def step(self):
        if self.out.shape[0]:
            for ph in self.PHASES:
                getattr(self, ph)()
