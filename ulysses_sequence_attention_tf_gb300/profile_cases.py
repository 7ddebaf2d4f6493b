"""Small, self-contained launches of one library kernel each, for profilers
(ncu captures one launch of a case run a few times).

  python -m ulysses_sequence_attention_tf_gb300.profile_cases projection [--S 8192] [--iters 3]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases scatter_fused [--S 32760] [--iters 3]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases scatter_fused_qk [--S 32760] [--iters 3]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases scatter --S 4096 --H 24 --layout fused
  python -m ulysses_sequence_attention_tf_gb300.profile_cases gather --P 8 --H 48 --D 64 --B 2 --S 6008
  python -m ulysses_sequence_attention_tf_gb300.profile_cases rope_table [--S 32760] [--iters 3]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases attention --P 1 --H 5 [--S 8192] [--softcap 50] [--docs 5]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases attention_backward --P 1 --H 5 [--S 8192] [--alibi]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases kv_append [--S 32760] [--tokens 4680] [--page 64]
  python -m ulysses_sequence_attention_tf_gb300.profile_cases kv_attend --B 24 --P 1 --H 16 --Hkv 4 --page 128

``--layout``: v_strided (Q/K contiguous, V a view into a fused projection; the
default), fused (Q/K/V all views of one fused projection), contiguous, pad16
(every head row followed by 16 bytes of padding: sources only 16-byte aligned,
which sends fused scatters to the register kernel).  ``rope_table`` builds the
resident cos/sin table of (theta, S, D) once per iteration, each time for
another theta.  ``attention`` and ``attention_backward`` see every key (``--alibi``: causal, with
distances as a bias; ``--docs``: within documents); the ``kv`` cases have --B sequences of --S tokens, the last --tokens of them new.

Inputs are the seeded synthetic ones of ``synth``; shapes default to the
video-DiT workload's head geometry (P=4, H=40, D=128, bf16) with a smaller
sequence for the projection, so a capture holds well under a few GB.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, build, synth


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("case", choices=["projection", "scatter", "scatter_fused", "scatter_fused_qk", "gather",
                                     "rope_table", "attention", "attention_backward", "kv_append", "kv_attend"])
    ap.add_argument("--P", type=int, default=4)
    ap.add_argument("--B", type=int, default=1)
    ap.add_argument("--D", type=int, default=128)
    ap.add_argument("--S", type=int, default=None, help="global tokens (default 8192 projection, 32760 others)")
    ap.add_argument("--H", type=int, default=40)
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--rope", choices=["interleaved", "neox"], default="interleaved")
    ap.add_argument("--layout", choices=["v_strided", "fused", "contiguous", "pad16"], default="v_strided")
    ap.add_argument("--dtype", choices=["bf16", "fp16"], default="bf16", help="element type of the scatters")
    ap.add_argument("--Hkv", type=int, default=None, help="key heads of the attention and cache cases (default H)")
    ap.add_argument("--softcap", type=float, default=0.0)
    ap.add_argument("--alibi", action="store_true")
    ap.add_argument("--docs", type=int, default=0, help="documents of unequal length in every batch row of the attention cases")
    ap.add_argument("--tokens", type=int, default=None, help="new tokens of a sequence (default 4680 kv_append, 1 kv_attend)")
    ap.add_argument("--page", type=int, default=64)
    args = ap.parse_args(argv)
    P, H, D, B = args.P, args.H, args.D, args.B
    S = args.S or (8192 if args.case in ("projection", "attention", "attention_backward") else 32760)
    Hkv = args.Hkv or H
    Sl, Hl = S // P, H // P
    build.build()
    binding.lib()
    binding.use_torch_allocator(True)
    dev = torch.device("cuda", 0)
    dt = torch.float16 if args.dtype == "fp16" and args.case != "projection" else torch.bfloat16
    wq, wk = synth.norm_weights(D, dt, seed=0, device=dev)
    if args.case == "projection":
        xs, w = synth.projection_inputs(P, B, Sl, H * D, H, D, torch.bfloat16, seed=1, device=dev)
        outs = {k: [torch.empty((B, S, Hl, D), dtype=torch.bfloat16, device=dev) for _ in range(P)] for k in "qkv"}

        def call():
            binding.project_qkv_into(xs, w, H, outs["q"], outs["k"], outs["v"], norm_rope=True, q_weight=wq,
                                     k_weight=wk, rope=args.rope)
    elif args.case == "rope_table":
        it = iter(range(args.iters))

        def call():
            binding.rope_table(10000.0 + next(it), S, D)
    elif args.case in ("attention", "attention_backward"):
        def rows(heads, seed):
            gen = torch.Generator(device=dev).manual_seed(seed)
            return [torch.randn((B, S, heads // P, D), generator=gen, device=dev).to(dt) for _ in range(P)]
        q, k, v, dout = rows(H, 0), rows(Hkv, 1), rows(Hkv, 2), rows(H, 3)
        kw = dict(softcap=args.softcap, causal=args.alibi)
        if args.alibi:
            kw["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev) / H)
        if args.docs:
            parts = [1 + 7 * i % 5 for i in range(args.docs)]
            ends = [S * sum(parts[:i]) // sum(parts) for i in range(1, args.docs)]
            docs = torch.bucketize(torch.arange(S, device=dev), torch.tensor(ends, device=dev), right=True).to(torch.int32)
            kw.update(q_docs=docs.expand(B, S).contiguous(), k_docs=docs.expand(B, S).contiguous())
        out, lse = binding.attention(q, k, v, **kw)

        def call():
            if args.case == "attention":
                binding.attention(q, k, v, out, lse, **kw)
            else:
                binding.attention_backward(dout, q, k, v, out, lse, **kw)
    elif args.case in ("kv_append", "kv_attend"):
        n = args.tokens or (4680 if args.case == "kv_append" else 1)
        used = -(-S // args.page)
        gen = torch.Generator(device=dev).manual_seed(0)
        cache = binding.kv_cache(B * used, Hkv, args.page, D, device=dev)
        for codes in cache[:2]:  # any finite codes
            codes.view(torch.uint8).random_(0, 0x70, generator=gen)
        where = (torch.randperm(B * used, generator=gen, device=dev).to(torch.int32).view(B, used),
                 torch.full((B,), S, dtype=torch.int32, device=dev),
                 torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev))
        q, k, v = ([torch.randn((B * n, heads // P, D), generator=gen, device=dev).to(dt) for _ in range(P)]
                   for heads in (H, Hkv, Hkv))
        q_out = [torch.empty_like(t) for t in q]

        def call():
            if args.case == "kv_append":
                binding.kv_append(cache, *where, k, v, q, q_out, q_weight=wq, k_weight=wk, rope=args.rope)
            else:
                binding.kv_attend(cache, *where, q, q_out, max_tokens=n, max_len=S, softcap=args.softcap, causal=n == 1)
    elif args.case in ("scatter", "scatter_fused", "scatter_fused_qk"):
        if args.layout == "pad16":
            pad = 16 // 2
            g = {key: [synth.qkv_shards(1, B, Sl, H, D + pad, dt, seed=10 * r + i, device=dev,
                                        with_k=False, with_v=False)["q"][0][..., :D] for r in range(P)]
                 for i, key in enumerate("qkv")}
        else:
            g = synth.qkv_shards(P, B, Sl, H, D, dt, seed=0, layout=args.layout, device=dev)
        v = None if args.case == "scatter_fused_qk" else g["v"]  # Q/K only: V moves elsewhere
        fused = args.case != "scatter"

        def call():
            if fused:
                binding.scatter_qkv("profile", g["q"], g["k"], v, norm_rope=True, q_weight=wq, k_weight=wk,
                                    rope=args.rope)
            else:
                binding.scatter_qkv("profile", g["q"], g["k"], v)
    else:
        attn = synth.attn_outputs(P, B, S, Hl, D, torch.bfloat16, seed=0, device=dev)

        def call():
            binding.gather_out("profile", attn)
    for _ in range(args.iters):
        call()
    torch.cuda.synchronize()
    print(f"{args.case}: {args.iters} launches, device status {binding.device_status()}")


if __name__ == "__main__":
    main()
