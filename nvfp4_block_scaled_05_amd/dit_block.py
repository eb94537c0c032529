"""The linear layers of one DiT (FLUX.2-style double-stream) block as an
NVFP4-patched model runs them, with every buffer allocated up front so the
sequence can be captured in a HIP graph and replayed.

Which layer runs in NVFP4 is decided by the exclude-pattern predicate
("英伟达B200狂飙10.2倍！AI绘图告别龟速！", nmedialink.com, section
"NVFP4量化"): the modulation linear on the timestep embedding contains
"stream" in its name and stays bf16; the attention projections and the MLP
are NVFP4 with weights quantized once at construction (quantize_weights=True)
and activations quantized dynamically on every call.  The MLP's hidden
activation is quantized with the amax the up-projection epilogue produced, so
it is read once.  Attention itself is not part of DitBlockLinears: the output
projection takes its input from the caller.  DitCrossBlock is a whole block
whose image tokens attend to a text encoder's states.
"""

import math

from . import (_device, _tensor, cache_attention, cache_attention_workspace, cache_write,
               cross_attention, cross_attention_workspace, gated_norm, gemm, gemm_bf16,
               gemm_workspace, kv_cache, layer_is_quantized, lora_add, lora_workspace, quantize,
               quantize_workspace, quantize_weight, rotary)

#: layer name -> (input, weight, epilogue)
LAYERS = {
    "double_stream_modulation_img.linear": ("temb", "w_mod", "none"),
    "transformer_blocks.0.attn.to_qkv": ("x_qkv", "w_qkv", "none"),
    "transformer_blocks.0.attn.to_out.0": ("x_o", "w_o", "none"),
    "transformer_blocks.0.ff.net.0.proj": ("x_mlp", "w_up", "gelu"),
    "transformer_blocks.0.ff.net.2": ("h", "w_down", "none"),
}


def gemm_flops(shapes):
    """2*M*N*K per layer for {input name: (rows, cols)} and the weights."""
    return {name: 2 * shapes[x][0] * shapes[w][0] * shapes[x][1]
            for name, (x, w, _) in LAYERS.items()}


class DitBlockLinears:
    """``weights``: bf16 device tensors w_mod, w_qkv, w_o, w_up, w_down
    ([out, in]); ``tokens``: rows of the token activations; ``cond_rows``:
    rows of the timestep embedding."""

    def __init__(self, weights, tokens, cond_rows=2):
        import torch
        dev = weights["w_qkv"].device
        self.quantized = {name: layer_is_quantized(name) for name in LAYERS}
        self.weights = {}
        for name, (_, w, _) in LAYERS.items():
            self.weights[name] = quantize_weight(weights[w]) if self.quantized[name] else weights[w]
        rows = {"temb": cond_rows, "x_qkv": tokens, "x_o": tokens, "x_mlp": tokens, "h": tokens}
        self.out = {}
        self.qbuf = {}
        self.ws = {}
        for name, (x, w, _) in LAYERS.items():
            n, k = weights[w].shape
            self.out[name] = torch.empty((rows[x], n), dtype=torch.bfloat16, device=dev)
            if self.quantized[name]:
                self.qbuf[name] = (torch.empty((rows[x], k // 2), dtype=torch.uint8, device=dev),
                                   torch.empty((rows[x], k // 16), dtype=torch.uint8, device=dev),
                                   torch.empty((1,), dtype=torch.float32, device=dev))
                self.ws[name] = gemm_workspace(rows[x], n, k, device=dev)
        self.amax = torch.empty((1,), dtype=torch.float32, device=dev)
        self.quant_ws = quantize_workspace(dev)
        names = list(LAYERS)
        # the up projection's epilogue amax feeds the down projection's quantize
        self.chain = self.quantized[names[3]] and self.quantized[names[4]]

    def _linear(self, name, x, amax_in=None, amax_out=None):
        epilogue = LAYERS[name][2]
        if not self.quantized[name]:
            return gemm_bf16(x, self.weights[name], epilogue=epilogue, out=self.out[name])
        q = quantize(x, amax=amax_in, workspace=None if amax_in is not None else self.quant_ws,
                     out=self.qbuf[name])
        return gemm(q, self.weights[name], epilogue=epilogue, y_amax=amax_out,
                    out=self.out[name], workspace=self.ws[name])

    def __call__(self, temb, x_qkv, x_o, x_mlp):
        names = list(LAYERS)
        self._linear(names[0], temb)
        self._linear(names[1], x_qkv)
        self._linear(names[2], x_o)
        amax = self.amax if self.chain else None
        h = self._linear(names[3], x_mlp, amax_out=amax)
        self._linear(names[4], h, amax_in=amax)
        return self.out


#: layer name -> (weight, epilogue) of DitCrossBlock
CROSS_LAYERS = {
    "double_stream_modulation_img.linear": ("w_mod", "none"),
    "transformer_blocks.0.attn.to_q": ("w_q", "none"),
    "transformer_blocks.0.attn.add_kv_proj": ("w_kv", "none"),
    "transformer_blocks.0.attn.to_out.0": ("w_o", "none"),
    "transformer_blocks.0.ff.net.0.proj": ("w_up", "gelu"),
    "transformer_blocks.0.ff.net.2": ("w_down", "none"),
}


class DitCrossBlock:
    """One block over image tokens that attend to a text encoder's states:

        h = norm(x) (1 + scale_a) + shift_a;     q = rotary(qk_norm(to_q(h)))
        r = x + gate_a to_out(attention(q, k, v))
        out = r + gate_m ff(norm(r) (1 + scale_m) + shift_m)

    with shift_a, scale_a, gate_a, shift_m, scale_m, gate_m the six parts of the
    modulation linear's output, and k, v made once per prompt by ``encode`` and
    kept over the denoising steps.  Linears run as in DitBlockLinears, every
    NVFP4 activation quantized with the amax its producer computed where that is
    one of these operators; all buffers are allocated here, so a call can be
    captured in a HIP graph.

    ``weights``: bf16 device tensors, [out, in]: w_mod [6 hidden, cond], w_q
    [heads * dim, hidden], w_kv [2 * kv_heads * dim, encoder width] (keys, then
    values), w_o, w_up, w_down.  ``q_norm`` / ``k_norm``: float32 [dim].
    ``plan``: a rotary plan for the image positions (text states carry none).
    ``lora``: layer name -> (down, up, scales), the adapters of all requests;
    ``ids`` of a call says which one each token uses.
    ``held``: "bf16", the prompts' keys and values as the projection and rotary leave
    them, or "nvfp4", in a cache of 4-bit codes (``cache``, a page for each prompt):
    9/32 of their memory, which every block of a model takes for every prompt over all
    steps.  Their bf16 form passes through the buffer of the MLP's hidden activations,
    which is made larger where it is too small for them, and is not kept: ``k`` and
    ``v`` are None.  Keys are quantized under the bound that their norm gives,
    sqrt(dim) max |k_norm|, values under the amax that the projection's epilogue
    computes (so that layer has to be one that runs in NVFP4).  The attention is of
    what 4 bits hold of them, and takes a fifth longer than over bf16 (2 x 16384
    queries of 512 and 77 states, 24 heads of 128: 207 us).
    """

    def __init__(self, weights, batch, tokens, states, heads, kv_heads, q_norm, k_norm, plan,
                 lora=None, held="bf16"):
        import torch
        if held not in ("bf16", "nvfp4"):
            raise ValueError(f"held must be 'bf16' or 'nvfp4', got {held!r}")
        dev = weights["w_q"].device
        self.batch, self.tokens, self.states = batch, tokens, states
        self.heads, self.kv_heads = heads, kv_heads
        self.q_norm, self.k_norm, self.plan = q_norm, k_norm, plan
        self.lora = dict(lora or {})
        self.mod, self.to_q, self.to_kv, self.to_out, self.up, self.down = CROSS_LAYERS
        unknown = set(self.lora) - {self.to_q, self.to_out, self.up, self.down}
        if unknown:
            raise ValueError(f"lora: not layers over the image tokens: {sorted(unknown)}")
        self.quantized = {name: layer_is_quantized(name) for name in CROSS_LAYERS}
        if held == "nvfp4" and not self.quantized[self.to_kv]:
            # (the bf16 passthrough computes no amax)
            raise ValueError(f"held='nvfp4' needs {self.to_kv} in NVFP4: its epilogue gives the values' amax")
        self.weights, self.out, self.qbuf, self.ws, self.lora_ws = {}, {}, {}, {}, {}

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)

        for name, (w, _) in CROSS_LAYERS.items():
            n, k = weights[w].shape
            rows = {"w_mod": batch, "w_kv": batch * states}.get(w, batch * tokens)
            self.weights[name] = quantize_weight(weights[w]) if self.quantized[name] else weights[w]
            self.out[name] = bf16(rows, n)
            if self.quantized[name]:
                self.qbuf[name] = (torch.empty((rows, k // 2), dtype=torch.uint8, device=dev),
                                   torch.empty((rows, k // 16), dtype=torch.uint8, device=dev),
                                   torch.empty((1,), dtype=torch.float32, device=dev))
                self.ws[name] = gemm_workspace(rows, n, k, device=dev)
            if name in self.lora:
                self.lora_ws[name] = lora_workspace(rows, k, self.lora[name][0].shape[1], device=dev)
        hidden = weights["w_q"].shape[1]
        dim = weights["w_q"].shape[0] // heads
        self.h, self.r = bf16(batch, tokens, hidden), bf16(batch, tokens, hidden)
        self.result = bf16(batch, tokens, hidden)
        self.attended = bf16(batch, tokens, heads, dim)
        self.k = self.v = None
        self.encoded = False
        # the block's own, so that a captured call finds the last prompt's lengths in it
        self.lengths = torch.full((batch,), states, dtype=torch.int32, device=dev)
        self.cache = None
        if held == "nvfp4":
            # no step needs the hidden activations of the one before, so a prompt may come
            # between any two
            kv, up = self.out[self.to_kv], self.out[self.up]
            shared = bf16(max(kv.numel(), up.numel()))
            self.out[self.to_kv] = shared[:kv.numel()].view(kv.shape)
            self.out[self.up] = shared[:up.numel()].view(up.shape)
            page = -(-states // 16) * 16
            bound = math.sqrt(dim) * float(k_norm.abs().max()) or 1.0
            self.cache = kv_cache(batch, page, kv_heads, dim, k_amax=bound, device=dev)
            self.first = torch.zeros((batch,), dtype=torch.int32, device=dev)
            self.attn_ws = cache_attention_workspace(batch, tokens, heads, kv_heads, dim, page, dev)
        else:
            self.attn_ws = cross_attention_workspace(batch, tokens, states, heads, kv_heads, dim, dev)
        self.amax = torch.zeros((1,), dtype=torch.float32, device=dev)
        self.quant_ws = quantize_workspace(dev)
        axes = (plan.axes,) if plan.axes > 1 else ()
        self.no_positions = torch.zeros((batch, states, *axes), dtype=torch.int32, device=dev)

    def _linear(self, name, x, ids=None, amax_in=None, amax_out=None):
        epilogue, out = CROSS_LAYERS[name][1], self.out[name]
        adapters = self.lora.get(name) if ids is not None else None
        own = "none" if adapters else epilogue
        if self.quantized[name]:
            q = quantize(x, amax=amax_in, workspace=None if amax_in is not None else self.quant_ws,
                         out=self.qbuf[name])
            gemm(q, self.weights[name], epilogue=own, y_amax=None if adapters else amax_out, out=out,
                 workspace=self.ws[name])
        else:
            gemm_bf16(x, self.weights[name], epilogue=own, out=out)
        if adapters:
            down, up, scales = adapters
            lora_add(out, x, down, up, ids, scales=scales, epilogue=epilogue, y_amax=amax_out,
                     workspace=self.lora_ws[name])
        return out

    def encode(self, states, lengths=None):
        """Keys and values of encoder ``states`` [batch, states, width] (bf16);
        ``lengths``: int32 [batch], the states of each prompt, None for all of
        them.  The rest is padding; it is quantized with the states, so it has to
        be finite.  All of it, the lengths too, is copied into the block's buffers:
        a captured call that is replayed after another prompt follows that one."""
        import torch
        if lengths is not None:
            _tensor(lengths, "lengths", torch.int32, (self.batch,))
            _device(states=states, lengths=lengths)
        # the amax of keys and values together bounds the values'
        amax = self.cache.amax[1:] if self.cache else None
        kv = self._linear(self.to_kv, states.view(-1, states.shape[-1]), amax_out=amax)
        kv = kv.view(self.batch, self.states, 2, self.kv_heads, -1)
        k, v = kv[:, :, 0], kv[:, :, 1]
        # text states carry no position: position 0, without the factor on rotated
        # values that a YaRN plan has, leaves their norm alone
        k = rotary(k, self.no_positions, self.plan._replace(magnitude=1.0), q_weight=self.k_norm, out=k)
        if self.cache:
            cache_write(self.cache, k, v, self.first)
        else:
            self.k, self.v = k, v
        self.encoded = True
        if lengths is None:
            self.lengths.fill_(self.states)
        else:
            self.lengths.copy_(lengths)

    def __call__(self, temb, x, positions, ids=None):
        """temb [batch, cond], x [batch, tokens, hidden], positions as ``rotary``
        takes them, ids: int32 [batch * tokens] or None (no adapters).  Returns
        [batch, tokens, hidden], overwritten by the next call."""
        if not self.encoded:
            raise ValueError("encode a prompt first")
        mod = self._linear(self.mod, temb)
        shift_a, scale_a, gate_a, shift_m, scale_m, gate_m = mod.chunk(6, 1)
        b, t, hidden = x.shape
        gated_norm(x, scale=scale_a, shift=shift_a, amax=self.amax, out=self.h)
        q = self._linear(self.to_q, self.h.view(b * t, hidden), ids, amax_in=self._given(self.to_q))
        q = q.view(b, t, self.heads, -1)
        rotary(q, positions, self.plan, q_weight=self.q_norm, out=q)
        if self.cache:
            cache_attention(q, self.cache, self.lengths, out=self.attended, workspace=self.attn_ws)
        else:
            cross_attention(q, self.k, self.v, kv_lengths=self.lengths, out=self.attended,
                            workspace=self.attn_ws)
        o = self._linear(self.to_out, self.attended.view(b * t, -1), ids)
        gated_norm(x, o.view(b, t, hidden), gate=gate_a, scale=scale_m, shift=shift_m,
                   amax=self.amax, residual_out=self.r, out=self.h)
        # the bf16 passthrough computes no amax; the adapters' kernel does
        has_amax = self.quantized[self.up] or (ids is not None and self.up in self.lora)
        chained = self._given(self.down) if has_amax else None
        u = self._linear(self.up, self.h.view(b * t, hidden), ids, amax_in=self._given(self.up),
                         amax_out=chained)
        d = self._linear(self.down, u, ids, amax_in=chained)
        gated_norm(self.r, d.view(b, t, hidden), gate=gate_m, norm=None, residual_out=self.result)
        return self.result

    def _given(self, name):
        """The amax word, where the layer quantizes its input with a producer's."""
        return self.amax if self.quantized[name] else None
