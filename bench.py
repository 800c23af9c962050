"""Benchmark of the fused equivariant convolution, forward + backward, on one
MI355X (gfx950).

Workload (default): the MACE-like large system -- 64,000 atoms uniform in a
cube at 0.1 atoms/A^3 (86.18 A side), 5 A cutoff (3,140,252 directed edges
for seed 0), node irreps 128x(0e+1o), harmonics up to l = 3, output
128x(0e+1o+2e+3o), 10 paths, per-edge per-path per-channel weights N(0,1),
upstream gradient N(0,1); fp32 storage.  Inputs are generated by
clebsch_gordan_tensor_amd.synth and sit in HBM before timing starts.

One step = e3_conv_forward + e3_conv_backward on the same graph (the
transposed edge index is prepared once per graph, timed separately).
`value` is edges/s over the K timed steps (wall clock between two device
synchronisations).  Every kernel is also timed with the pages' protocol
(e3j 3.1: warm-ups, then 100 individually timed launches; median, minimum
and mean of the fastest 20%).
Side measurements (in "kernels", outside the step): the chain from the
harmonic cotangent dY to per-atom position gradients on the same graph, the
batched tensor product forward and backward on its 200,000-row workload, the
per-irrep channel mixing on the matrix cores, the normalisation and the
clipped AdamW step, and the radial-MLP forms.
"configs": the other convolution workloads (tiny 64-atom, water3k 3,000-atom
with radial-MLP weights, ho20k 20,000-atom bf16 with 23 paths), each with
algorithmic bytes and the method's flops against the HBM and fp32 VALU peaks
(and cold-cache runs where the node rows fit the Infinity Cache).
Printed: one JSON line with edges/s (value), the per-kernel times, the
roofline of the dominant kernel (algorithmic bytes of the e3j paper's Eq.9 /
measured duration, against the 8 TB/s HBM peak, and against the rate torch's
own streaming kernels reach for the same read:write mix) and the fp64 CPU
oracle timed on bounded samples (all threads; water3k also on one thread).
"""
from __future__ import annotations

import argparse
import json
import os
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

HBM_PEAK_GBS = 8000.0
TRAFFIC_FILE = os.path.join(ROOT, "profiles", "conv_bwd_mace64k_traffic.txt")


# sources the convolution kernels are built from (not the channel mixing)
# the sources the profiled convolution kernels (mace64k signature) are built
# from, and the prepare step whose node order sets their gathers' reuse
_CONV_SOURCES = ("kernels/common.h", "kernels/conv_kernels.h", "kernels/signatures.h",
                 "kernels/inst_l1to3.hip", "kernels/prep.hip", "host/cg_ladder.h",
                 "host/cg_ladder.cpp", "host/gen_cg_table.cpp")


def kernel_sources_sha1() -> str:
    """Hash of the convolution kernels' sources: counter-measured traffic only
    applies to the kernels it was measured on."""
    import hashlib
    h = hashlib.sha1()
    base = os.path.join(ROOT, "clebsch_gordan_tensor_amd", "csrc")
    for rel in _CONV_SOURCES:
        with open(os.path.join(base, rel), "rb") as f:
            h.update(rel.encode())
            h.update(f.read())
    return h.hexdigest()


def measured_traffic(config: str):
    """HBM bytes per backward launch from the committed counter summary, if
    it was taken on this workload with these kernel sources (else None)."""
    if not os.path.exists(TRAFFIC_FILE):
        return None
    kv = {}
    with open(TRAFFIC_FILE) as f:
        for line in f:
            if ":" in line and not line.lstrip().startswith("#"):
                k, v = line.split(":", 1)
                kv[k.strip()] = v.strip()
    if kv.get("workload") != config or kv.get("kernel_sources_sha1") != kernel_sources_sha1():
        return None
    try:
        return {"total": float(kv["conv_backward_hbm_bytes_per_launch"]),
                "read": float(kv["conv_backward_hbm_read_bytes_per_launch"]),
                "write": float(kv["conv_backward_hbm_write_bytes_per_launch"])}
    except (KeyError, ValueError):
        return None
CPU_SAMPLE_RECEIVERS = 64000


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def algorithmic_bytes(N, E, dx, dy, dout, P, C, esize):
    """Eq.9 of the e3j paper: sizeof(inputs) + sizeof(outputs); the backward
    counts primals, the output cotangent and the input cotangents; int32
    index arrays included."""
    x = N * dx * C * esize
    w = E * P * C * esize
    ev = E * 3 * 4
    m = N * dout * C * esize
    fwd = x + w + ev + m + (N + 1) * 4 + E * 4
    bwd = x + w + ev + m + x + w + E * dy * 4 + (N + 1) * 4 + 2 * E * 4
    return fwd, bwd


def cpu_baseline(p, n_recv):
    """fp64 oracle on a bounded sample: the in-edges of n_recv receivers
    (forward and edge cotangents) and the out-edges of the same nodes as
    senders (node cotangent)."""
    from clebsch_gordan_tensor_amd.synth import edges_of_receivers, edges_of_senders
    from oracle import oracle as O

    g = p.graph
    od = O.Desc(p.x_irreps, p.y_irreps, p.out_irreps, p.channels)
    rng = np.random.default_rng(7)
    nodes = np.sort(rng.choice(g.n_nodes, min(n_recv, g.n_nodes), replace=False))
    rp, sn, ev, ids = edges_of_receivers(g, nodes)
    rp2, sn2, ev2, ids2 = edges_of_senders(g, nodes)
    x64 = p.x.astype(np.float64)
    w_in, w_out = p.w[ids].astype(np.float64), p.w[ids2].astype(np.float64)
    dm64 = p.dm.astype(np.float64)
    t0 = time.perf_counter()
    O.conv_forward(od, rp, sn, x64, w_in, evec=ev, rows=nodes)
    O.conv_backward_edge(od, rp, sn, x64, w_in, dm64, evec=ev)
    O.conv_backward_dx(od, rp2, sn2, w_out, dm64, evec=ev2, rows=nodes)
    dt = time.perf_counter() - t0
    return {"value": len(ids) / dt, "unit": "edges/s", "cores": O.num_threads(),
            "kind": "oracle",
            "sample": f"{len(nodes)} random receivers of the same graph: forward and dw/dY over "
                      f"their {len(ids)} in-edges, dx over the same nodes as senders "
                      f"({len(ids2)} out-edges); fp64, {dt:.2f} s"}


def protocol(fn, stream, runs=100, warm=10, between=None):
    """The pages' timing protocol (e3j 3.1 unit benchmarks): warm-up launches,
    then `runs` launches each bracketed by its own HIP events on the launch
    stream; median, minimum and the mean of the fastest 20%.  `between` (not
    timed) runs before each timed launch, e.g. to evict the caches."""
    import torch
    for _ in range(warm):
        fn()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
          for _ in range(runs)]
    for a, b in ev:
        if between is not None:
            between()
        a.record(stream)
        fn()
        b.record(stream)
    torch.cuda.synchronize()
    t = np.sort(np.array([a.elapsed_time(b) for a, b in ev]))
    k = max(1, runs // 5)
    return {"ms": float(np.median(t)), "median_ms": float(np.median(t)), "min_ms": float(t[0]),
            "fastest20_mean_ms": float(t[:k].mean()), "mean_ms": float(t.mean()), "runs": runs}


def time_call(fn, stream, reps):
    """Per-launch statistics of fn() (the protocol above, `reps` runs)."""
    return protocol(fn, stream, runs=reps, warm=2)


def tp_measurements(api, S, dev, stream):
    """Batched tensor product forward and backward on the 200k-row workload
    (x 128x(0e+1o+2e), y harmonics l <= 3, out 128x(0e+1o+2e+3o), 17 paths)."""
    import torch
    t0 = time.time()
    q = S.make_tp(with_dz=True)
    B, C = q.x.shape[0], q.channels
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    x, w, dz, u = up(q.x), up(q.w), up(q.dz), up(q.u)
    del q.x, q.w, q.dz
    d = api.Desc(q.x_irreps, q.y_irreps, q.out_irreps, C)
    P = api.num_paths(d)
    y = api.spherical_harmonics(3, u)
    z = torch.empty((B, d.dout, C), device=dev, dtype=torch.float32)
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    dy = torch.empty((B, d.dy), device=dev, dtype=torch.float32)
    log(f"[bench] tensor product: {B} rows (generated in {time.time() - t0:.1f} s)")
    f = time_call(lambda: api.tp_forward(d, x, y, w, out=z), stream, 100)
    b = time_call(lambda: api.tp_backward(d, x, y, w, dz, dx=dx, dw=dw, dy=dy), stream, 100)
    fb = B * 4 * ((d.dx + P + d.dout) * C + d.dy)
    bb = B * 4 * ((2 * d.dx + 2 * P + d.dout) * C + 2 * d.dy)
    for r, nb in ((f, fb), (b, bb)):
        r["bytes"] = nb
        r["gbs"] = nb / (r["ms"] * 1e-3) / 1e9
        r["frac"] = r["gbs"] / HBM_PEAK_GBS
        r["rows_per_s"] = B / (r["ms"] * 1e-3)
    log(f"[bench] tp forward {f['ms']:.3f} ms ({f['gbs']:.0f} GB/s), "
        f"backward {b['ms']:.3f} ms ({b['gbs']:.0f} GB/s)")
    return {"tp_forward_200k": f, "tp_backward_200k": b}


MFMA_F32_PEAK_TFLOPS = 157.3


def linear_measurement(api, S, p, dev, stream):
    """Per-irrep channel mixing of the workload's output features (Cout = Cin
    = C, one C x C matrix per irrep) on the fp32 matrix cores."""
    import torch
    ins = outs = p.out_irreps
    N, C = p.graph.n_nodes, p.channels
    d = S.dim(ins)
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn((N, d, C), device=dev, generator=g)
    W = torch.randn((api.linear_num_weights(ins, outs), C, C), device=dev, generator=g) / C ** 0.5
    y = torch.empty_like(x)
    r = time_call(lambda: api.linear(ins, outs, x, W, out=y), stream, 100)
    flops = 2.0 * N * d * C * C
    r["bytes"] = 2 * x.numel() * 4 + W.numel() * 4
    r["tflops"] = flops / (r["ms"] * 1e-3) / 1e12
    r["frac_mfma_f32"] = r["tflops"] / MFMA_F32_PEAK_TFLOPS
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    dx, dW = api.linear_backward(ins, outs, x, W, y, dx=dx, dW=dW)
    b = time_call(lambda: api.linear_backward(ins, outs, x, W, y, dx=dx, dW=dW), stream, 100)
    b["tflops"] = 2 * flops / (b["ms"] * 1e-3) / 1e12
    b["frac_mfma_f32"] = b["tflops"] / MFMA_F32_PEAK_TFLOPS
    log(f"[bench] channel mixing {N}x{d}x{C}: forward {r['ms']*1e3:.1f} us "
        f"({r['tflops']:.1f} TFLOP/s), backward {b['ms']*1e3:.1f} us ({b['tflops']:.1f} TFLOP/s)")
    return {"linear_fp32_mfma": r, "linear_backward_fp32_mfma": b}


def training_measurement(api, S, p, dev, stream):
    """What training adds to the layers: the normalisation of the workload's
    output features with its gradients, and the clipped AdamW step over the
    weights of twelve layers (channel mixings, radial MLP, normalisations),
    moments in 32 and in 8 bits."""
    import torch
    ir, N, C = p.out_irreps, p.graph.n_nodes, p.channels
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn((N, S.dim(ir), C), device=dev, generator=g)
    dy = torch.randn((N, S.dim(ir), C), device=dev, generator=g)
    w, b = torch.ones((len(ir), C), device=dev), torch.zeros((1, C), device=dev)
    y, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(api.layer_norm_workspace_size(ir, N, C), device=dev, dtype=torch.uint8)
    f = time_call(lambda: api.layer_norm(ir, x, w, b, out=y), stream, 100)
    r = time_call(lambda: api.layer_norm_backward(ir, x, w, dy, dx=y, dweight=dw, dbias=db,
                                                  workspace=ws), stream, 100)
    for rec, n in ((f, 2), (r, 3)):
        rec["bytes"] = n * 4 * x.numel()
        rec["gbs"] = rec["bytes"] / (rec["ms"] * 1e-3) / 1e9
    del x, dy, y
    sizes = [len(ir) * C * C, 2 * C * C, 8 * 64, 64 * p.n_paths * C, len(ir) * C, C] * 12
    params = [torch.randn(n, device=dev, generator=g) for n in sizes]
    grads = [torch.randn(n, device=dev, generator=g) for n in sizes]
    out = {"layer_norm": f, "layer_norm_backward": r}
    for bits in (32, 8):
        m, v, ms, vs = api.adamw_state(params, bits)
        ps = api.Params(params, grads, m, v, m_scale=ms, v_scale=vs, weight_decay=0.01)

        def update():
            norm = api.grad_norm(ps, max_norm=1.0)
            api.adamw(ps, 1, 1e-4, grad_scale=norm[1:])

        out[f"clipped_adamw_{bits}bit"] = time_call(update, stream, 100)
        out[f"clipped_adamw_{bits}bit"]["elements"] = sum(sizes)
    log(f"[bench] normalisation {N}x{S.dim(ir)}x{C}: forward {f['ms']*1e3:.1f} us "
        f"({f['gbs']:.0f} GB/s), backward {r['ms']*1e3:.1f} us ({r['gbs']:.0f} GB/s); clipped AdamW "
        f"over {sum(sizes)} weights in {len(sizes)} tensors: "
        + ", ".join(f"{out[f'clipped_adamw_{k}bit']['ms']*1e3:.1f} us ({k}-bit moments)"
                    for k in (32, 8)))
    return out


MFMA_F16_PEAK_TFLOPS = 2500.0


def radial_measurement(api, d, g, rowptr, sender, ev, x, wbuf, ws, dev, stream):
    """The convolution with its weights from the radial MLP (8 Bessel functions
    -> 64 SiLU units -> P*C): fused (w never stored) against MLP-then-conv,
    on the same graph and features.  wbuf ([E][P][C] float32) is scratch."""
    import torch
    P, C = api.num_paths(d), d.channels
    gen = torch.Generator(device=dev).manual_seed(1)
    W1 = torch.randn((8, 64), device=dev, generator=gen) / 8 ** 0.5
    W2 = torch.randn((64, P * C), device=dev, generator=gen) / 8.0
    m = torch.empty((g.n_nodes, d.dout, C), device=dev, dtype=torch.float32)
    try:
        api.conv_forward_radial(d, rowptr, sender, ev, x, 5.0, W1, W2, out=m, workspace=ws)
    except api.E3Error:
        return {}
    fused = time_call(lambda: api.conv_forward_radial(d, rowptr, sender, ev, x, 5.0, W1, W2,
                                                      out=m, workspace=ws), stream, 100)
    # the hidden layer once per edge, then the convolution reading it
    hid = api.radial_hidden(ev, 5.0, W1, W2)
    hidden = time_call(lambda: api.radial_hidden(ev, 5.0, W1, W2, out=hid), stream, 100)
    fused_h = time_call(lambda: api.conv_forward_radial_hidden(d, rowptr, sender, ev, x, 5.0, W1,
                                                               W2, hid, out=m, workspace=ws),
                        stream, 100)

    def hidden_then_fused():
        api.radial_hidden(ev, 5.0, W1, W2, out=hid)
        api.conv_forward_radial_hidden(d, rowptr, sender, ev, x, 5.0, W1, W2, hid, out=m,
                                       workspace=ws)

    fused_h_total = time_call(hidden_then_fused, stream, 100)
    w2d = wbuf.view(g.n_edges, P * C)
    mlp_h = time_call(lambda: api.radial_mlp_hidden(hid, g.n_edges, 5.0, W1, W2, out=w2d),
                      stream, 50)
    # the backward: w formed again from the hidden layer inside the convolution
    # backward, against the MLP writing w and the convolution backward reading it
    dm = torch.randn((g.n_nodes, d.dout, C), device=dev, generator=gen)
    bdx = torch.empty((g.n_nodes, d.dx, C), device=dev, dtype=torch.float32)
    bdw = torch.empty((g.n_edges, P, C), device=dev, dtype=torch.float32)
    bdY = torch.empty((g.n_edges, d.dy), device=dev, dtype=torch.float32)
    scr = torch.empty(api.conv_backward_radial_scratch_bytes(d, g.n_edges), device=dev,
                      dtype=torch.uint8)
    bwd_f = time_call(lambda: api.conv_backward_radial_hidden(
        d, rowptr, sender, ws, ev, x, 5.0, W1, W2, hid, dm, dx=bdx, dw=bdw, dY=bdY, scratch=scr),
        stream, 50)

    def composed_bwd():
        api.radial_mlp_hidden(hid, g.n_edges, 5.0, W1, W2, out=w2d)
        api.conv_backward(d, rowptr, sender, ws, ev, x, wbuf, dm, dx=bdx, dw=bdw, dY=bdY)

    bwd_c = time_call(composed_bwd, stream, 50)
    del hid, scr, bdx, bdY, dm
    mlp = time_call(lambda: api.radial_mlp(ev, 5.0, W1, W2, out=w2d), stream, 50)

    def composed():
        api.radial_mlp(ev, 5.0, W1, W2, out=w2d)
        api.conv_forward(d, rowptr, sender, ev, x, wbuf, out=m, workspace=ws)

    comp = time_call(composed, stream, 50)
    # the MLP's backward for a cotangent of w's shape (w itself stands in)
    nb = api.radial_mlp_backward_workspace_bytes(W1, W2, g.n_edges, P * C)
    rws = torch.empty(nb, device=dev, dtype=torch.uint8)
    bwd = time_call(lambda: api.radial_mlp_backward(ev, 5.0, W1, W2, w2d, workspace=rws), stream, 50)
    E = g.n_edges
    mfma_flops = 3 * 2.0 * 64 * P * C * E  # three fp16 products per hidden unit and column
    fused["edges_per_s"] = E / (fused["ms"] * 1e-3)
    fused["mfma_tflops_f16"] = mfma_flops / (fused["ms"] * 1e-3) / 1e12
    fused["frac_mfma_f16"] = fused["mfma_tflops_f16"] / MFMA_F16_PEAK_TFLOPS
    mlp["bytes_written"] = E * P * C * 4
    mlp["gbs"] = mlp["bytes_written"] / (mlp["ms"] * 1e-3) / 1e9
    bwd["dw_bytes_read"] = E * P * C * 4  # once, for both products
    bwd["gbs_dw"] = bwd["dw_bytes_read"] / (bwd["ms"] * 1e-3) / 1e9
    log(f"[bench] radial conv forward: fused {fused['ms']:.3f} ms, hidden layer "
        f"{hidden['ms']:.3f} ms + fused reading it {fused_h['ms']:.3f} ms = "
        f"{fused_h_total['ms']:.3f} ms, MLP {mlp['ms']:.3f} ms (from the hidden layer "
        f"{mlp_h['ms']:.3f}) + conv = {comp['ms']:.3f} ms; "
        f"conv backward from the hidden layer {bwd_f['ms']:.3f} ms against MLP + conv "
        f"backward {bwd_c['ms']:.3f} ms; MLP backward {bwd['ms']:.3f} ms")
    return {"conv_forward_radial_fused": fused, "radial_hidden": hidden,
            "conv_forward_radial_hidden": fused_h,
            "radial_hidden_then_conv_forward_radial_hidden": fused_h_total,
            "radial_mlp": mlp, "radial_mlp_from_hidden": mlp_h,
            "radial_mlp_then_conv_forward": comp,
            "conv_backward_radial_hidden": bwd_f,
            "radial_mlp_from_hidden_then_conv_backward": bwd_c,
            "radial_mlp_backward": bwd}


def generic_sweep(L_list):
    """The coefficient-table and dense-product tensor product and convolution
    at degrees 1..8 on the workloads of e3j B.1: TP on 32,768 rows (Figs
    5-6), convolution on 2,048 atoms with about 45 neighbours (Fig 7), 128
    channels, every irrep 0..L once with parity (-1)^l, harmonics 0..L;
    inputs N(0,1) from a seeded device generator (timing only).  The table
    kernels hold at most 63 components per operand, so from L = 7 (64) only
    the dense products run; at L = 8 (81 harmonics per edge) the dense
    convolution forward takes the harmonics as an input.  One JSON line on
    stdout."""
    import torch

    from clebsch_gordan_tensor_amd import api
    from clebsch_gordan_tensor_amd import synth as S

    api.lib()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream()
    gen = torch.Generator(device=dev).manual_seed(0)
    g = S.random_graph(2048, 26.75, 5.0, 0)
    N, E, C, B = g.n_nodes, g.n_edges, 128, 32768
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    rowptr, sender, ev = up(g.rowptr), up(g.sender), up(g.evec)
    ws = api.conv_prepare_transpose(rowptr, sender, edge_vec=ev)
    log(f"[generic] graph N={N} E={E} ({E / N:.1f} neighbours), TP rows {B}, C={C}")
    rows = []
    for L in L_list:
        ir = S.degree_irreps(L)
        d = api.Desc(ir, S.sh_irreps(L), ir, C)
        P = api.num_paths(d)
        rn = lambda *shape: torch.randn(shape, device=dev, generator=gen)
        x, w, dz = rn(B, d.dx, C), rn(B, P, C), rn(B, d.dout, C)
        y = api.spherical_harmonics(L, rn(B, 3))
        z = torch.empty_like(dz)
        table = d.dx <= 63 and d.dout <= 63
        skip = {"ms": None}
        tf = time_call(lambda: api.tp_forward_generic(d, x, y, w, out=z), stream, 5) if table else skip
        tg = time_call(lambda: api.tp_forward_gemm(d, x, y, w, out=z), stream, 5)
        tb = time_call(lambda: api.tp_backward_generic(d, x, y, w, dz), stream, 3) if table else skip
        tbg = time_call(lambda: api.tp_backward_gemm(d, x, y, w, dz), stream, 5)
        del x, w, dz, y, z
        x, w, dm = rn(N, d.dx, C), rn(E, P, C), rn(N, d.dout, C)
        m = torch.empty_like(dm)
        cf = time_call(lambda: api.conv_forward_generic(d, rowptr, sender, ev, x, w, out=m,
                                                        workspace=ws), stream, 5) if table else skip
        cb = time_call(lambda: api.conv_backward_generic(d, rowptr, sender, ws, ev, x, w, dm),
                       stream, 3) if table else skip
        # the dense backward takes given harmonics, and so does the forward
        # past 64 harmonics per edge (L = 8)
        dg = api.Desc(ir, S.sh_irreps(L), ir, C, api.E3_Y_GIVEN)
        Yg = api.spherical_harmonics(L, ev)
        if d.dy <= 64:
            cg = time_call(lambda: api.conv_forward_gemm(d, rowptr, sender, ev, x, w, out=m),
                           stream, 5)
        else:
            cg = time_call(lambda: api.conv_forward_gemm(dg, rowptr, sender, Yg, x, w, out=m),
                           stream, 5)
        cbg = time_call(lambda: api.conv_backward_gemm(dg, rowptr, sender, ws, Yg, x, w, dm),
                        stream, 5)
        del x, w, dm, m, Yg
        r = {"L": L, "paths": P, "tp_forward_ms": tf["ms"], "tp_forward_gemm_ms": tg["ms"],
             "tp_backward_ms": tb["ms"], "tp_backward_gemm_ms": tbg["ms"],
             "conv_forward_ms": cf["ms"], "conv_forward_gemm_ms": cg["ms"],
             "conv_backward_ms": cb["ms"], "conv_backward_gemm_ms": cbg["ms"],
             "tp_forward_bytes": B * 4 * ((d.dx + P + d.dout) * C + d.dy),
             "conv_forward_bytes": 4 * (E * (P * C + 3 + 1) + N * (d.dx + d.dout) * C)}
        rows.append(r)
        f3 = lambda v: "-" if v is None else f"{v:.3f}"
        log(f"[generic] L={L} P={P}: TP fwd {f3(tf['ms'])} ms (dense products {tg['ms']:.3f}) "
            f"bwd {f3(tb['ms'])} ms (dense {tbg['ms']:.3f}) | "
            f"conv fwd {f3(cf['ms'])} ms (dense products {cg['ms']:.3f}) bwd {f3(cb['ms'])} ms "
            f"(dense {cbg['ms']:.3f})")
    print(json.dumps({"generic_sweep": rows, "graph_edges": E, "tp_rows": B, "channels": C}))


VALU_F32_PEAK_TFLOPS = 157.3          # published fp32 vector peak (packed FMA)
VALU_F32_NONPACKED_TFLOPS = 78.6      # 256 CUs x 4 SIMDs x 16 lanes x 2 flops x 2.4 GHz


def method_flops(api, d):
    """The method's own work per edge and channel (not a dense equivalent):
    forward 2 nnz + 2 sum_P (2L+1) (the CG products and the per-path
    weighting), backward 7 nnz + 4 sum_P (2L+1); nnz = the real CG blocks'
    non-zeros over all paths."""
    nnz = sum_l = 0
    for i in range(api.num_paths(d)):
        ix, iy, io = api.path_info(d, i)
        l1, l2, L = d.x[ix][0], d.y[iy][0], d.out[io][0]
        nnz += int((np.abs(api.cg_block(l1, l2, L)) > 1e-12).sum())
        sum_l += 2 * L + 1
    return 2 * nnz + 2 * sum_l, 7 * nnz + 4 * sum_l


def hbm_ceilings(dev, stream):
    """Achievable HBM rates with torch's own streaming kernels on 1 GiB
    buffers: read only (a sum), 1:1 (a copy) and 2:1 (an add)."""
    import torch
    n = 1 << 28
    a = torch.ones(n, device=dev)
    b = torch.ones(n, device=dev)
    c = torch.empty(n, device=dev)
    out = {}
    for name, fn, nbytes in (("read_gbs", lambda: torch.sum(a), 4 * n),
                             ("copy_gbs", lambda: c.copy_(a), 8 * n),
                             ("add_gbs", lambda: torch.add(a, b, out=c), 12 * n)):
        r = protocol(fn, stream, runs=20, warm=3)
        out[name] = nbytes / (r["median_ms"] * 1e-3) / 1e9
    del a, b, c
    return out


def mix_ceiling_gbs(read_bytes, write_bytes, ceil):
    """Rate of a read:write mix between 1:1 and 2:1 composed from the copy
    (1:1) and add (2:1) rates: W1 bytes copied, W2 added, with W1 + W2 = W
    and W1 + 2 W2 = R."""
    R, W = float(read_bytes), float(write_bytes)
    w2 = min(max(R - W, 0.0), W)
    w1 = W - w2
    t = 2 * w1 / (ceil["copy_gbs"] * 1e9) + 3 * w2 / (ceil["add_gbs"] * 1e9)
    return (w1 * 2 + w2 * 3) / t / 1e9


def conv_record(api, S, name, dev, stream, runs=100):
    """One workload of the configs as a sub-record: prepare, forward and
    backward under the timing protocol, algorithmic bytes (Eq.9) and the
    method's flops against the HBM and fp32 VALU peaks."""
    import torch
    t0 = time.time()
    p = S.make_conv(name)
    g = p.graph
    N, E, C, P = g.n_nodes, g.n_edges, p.channels, p.n_paths
    tdt = torch.bfloat16 if p.dtype == "bf16" else torch.float32
    up = lambda a, dt=None: (torch.from_numpy(np.ascontiguousarray(a)).to(dev)
                             if dt is None else torch.from_numpy(a).to(dev).to(dt))
    rowptr, sender, ev = up(g.rowptr), up(g.sender), up(g.evec)
    x, w, dm = up(p.x, tdt), up(p.w, tdt), up(p.dm, tdt)
    d = api.Desc(p.x_irreps, p.y_irreps, p.out_irreps, C)
    m = torch.empty((N, d.dout, C), device=dev, dtype=tdt)
    dxo, dwo = torch.empty_like(x), torch.empty_like(w)
    dYo = torch.empty((E, d.dy), device=dev, dtype=torch.float32)
    ws = torch.empty(api.workspace_size(N, E), device=dev, dtype=torch.uint8)
    prep = protocol(lambda: api.conv_prepare_transpose(rowptr, sender, ws, edge_vec=ev), stream,
                    runs=20, warm=2)
    fwd = protocol(lambda: api.conv_forward(d, rowptr, sender, ev, x, w, out=m, workspace=ws),
                   stream, runs=runs)
    bwd = protocol(lambda: api.conv_backward(d, rowptr, sender, ws, ev, x, w, dm, dx=dxo, dw=dwo,
                                             dY=dYo), stream, runs=runs)
    esize = 2 if p.dtype == "bf16" else 4
    fb, bb = algorithmic_bytes(N, E, d.dx, d.dy, d.dout, P, C, esize)
    ff, bf = method_flops(api, d)
    rec = {"workload": name, "n_nodes": N, "n_edges": E, "channels": C, "paths": P,
           "dtype": p.dtype, "prepare": prep}
    for key, r, nb, fl in (("forward", fwd, fb, ff), ("backward", bwd, bb, bf)):
        s_ = r["median_ms"] * 1e-3
        r.update(bytes=nb, gbs=nb / s_ / 1e9, hbm_frac=nb / s_ / 1e9 / HBM_PEAK_GBS,
                 flops=float(fl) * E * C, tflops=float(fl) * E * C / s_ / 1e12,
                 valu_frac=float(fl) * E * C / s_ / 1e12 / VALU_F32_PEAK_TFLOPS,
                 valu_frac_nonpacked=float(fl) * E * C / s_ / 1e12 / VALU_F32_NONPACKED_TFLOPS)
        rec[key] = r
    rec["edges_per_s_fwd_bwd"] = E / ((fwd["median_ms"] + bwd["median_ms"]) * 1e-3)
    # the dominant kernel against the peak of whichever unit it uses more of
    # (HBM bytes, or fp32 vector flops against the published peak; the kernels
    # are built without packed fp32, whose own peak is half: valu_frac_nonpacked)
    dom = "backward" if bwd["median_ms"] >= fwd["median_ms"] else "forward"
    rd = rec[dom]
    alu = rd["valu_frac"] > rd["hbm_frac"]
    rec["roofline"] = {"kernel": "conv_" + dom, "bound": "alu" if alu else "hbm",
                       "achieved": rd["tflops"] if alu else rd["gbs"],
                       "peak": VALU_F32_PEAK_TFLOPS if alu else HBM_PEAK_GBS,
                       "unit": "TFLOP/s" if alu else "GB/s",
                       "frac": rd["valu_frac"] if alu else rd["hbm_frac"], "traffic": None}
    if fb < (1 << 30):
        # node rows fit the 256 MB Infinity Cache: also cold, a 1 GiB fill between runs
        junk = torch.empty(1 << 28, device=dev)
        cold = lambda: junk.fill_(1.0)
        rec["forward_cold"] = protocol(lambda: api.conv_forward(d, rowptr, sender, ev, x, w, out=m,
                                                                workspace=ws),
                                       stream, runs=runs // 2, warm=2, between=cold)
        rec["backward_cold"] = protocol(lambda: api.conv_backward(d, rowptr, sender, ws, ev, x, w,
                                                                  dm, dx=dxo, dw=dwo, dY=dYo),
                                        stream, runs=runs // 2, warm=2, between=cold)
        del junk
    log(f"[bench] {name}: N={N} E={E} {p.dtype}: fwd {fwd['median_ms']:.3f} ms "
        f"({rec['forward']['gbs']:.0f} GB/s, {rec['forward']['tflops']:.1f} TFLOP/s), bwd "
        f"{bwd['median_ms']:.3f} ms ({rec['backward']['gbs']:.0f} GB/s, "
        f"{rec['backward']['tflops']:.1f} TFLOP/s), prepare {prep['median_ms']:.3f} ms "
        f"(set up in {time.time() - t0:.1f} s)")
    del x, w, dm, m, dxo, dwo, dYo, ws
    torch.cuda.empty_cache()
    return rec, p


def cpu_model() -> str:
    try:
        with open("/proc/cpuinfo") as f:
            for line in f:
                if line.startswith("model name"):
                    return line.split(":", 1)[1].strip()
    except OSError:
        pass
    return "unknown"


def cpu_full(p, threads=None):
    """The fp64 oracle over a whole (small) workload, forward and backward,
    optionally on a set number of threads; edges/s."""
    from oracle import oracle as O
    g = p.graph
    od = O.Desc(p.x_irreps, p.y_irreps, p.out_irreps, p.channels)
    n0 = O.num_threads()
    if threads:
        O.set_num_threads(threads)
    try:
        t0 = time.perf_counter()
        O.conv_forward(od, g.rowptr, g.sender, p.x, p.w, evec=g.evec)
        O.conv_backward_dx(od, g.rowptr, g.sender, p.w, p.dm, evec=g.evec)
        O.conv_backward_edge(od, g.rowptr, g.sender, p.x, p.w, p.dm, evec=g.evec)
        dt = time.perf_counter() - t0
        used = O.num_threads()
    finally:
        O.set_num_threads(n0)
    return {"value": g.n_edges / dt, "unit": "edges/s", "cores": used, "kind": "oracle",
            "sample": f"the whole {p.name} workload ({g.n_edges} edges), forward and backward, "
                      f"fp64, {dt:.2f} s"}


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--config", default="mace64k")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-extras", action="store_true",
                    help="skip the side measurements (force chain, tensor product)")
    ap.add_argument("--print-kernel-hash", action="store_true")
    ap.add_argument("--no-configs", action="store_true",
                    help="skip the other workloads' sub-records (tiny, water3k, ho20k)")
    ap.add_argument("--generic-sweep", default="",
                    help="only time the coefficient-table and dense-product paths at these degrees (e.g. 1,2,3,4,5,6,7,8)")
    ap.add_argument("--calibrate-copy", action="store_true",
                    help="only run a 4 GiB device-to-device copy (counter calibration)")
    args = ap.parse_args()
    if args.print_kernel_hash:
        print(kernel_sources_sha1())
        return
    if args.generic_sweep:
        generic_sweep([int(v) for v in args.generic_sweep.split(",")])
        return
    if args.calibrate_copy:
        import torch
        a = torch.empty(1 << 30, dtype=torch.float32, device="cuda:0")
        b = torch.empty_like(a)
        a.fill_(1.0)
        for _ in range(3):
            b.copy_(a)
        torch.cuda.synchronize()
        print(json.dumps({"copy_bytes_read": a.numel() * 4, "copy_bytes_written": b.numel() * 4}))
        return
    if args.gpus != 1:
        print("bench.py measures one GPU: there is no multi-GPU path (the convolution would "
              "shard by receiver ranges with a halo exchange of sender rows); use --gpus 1",
              file=sys.stderr)
        sys.exit(2)

    import torch

    from clebsch_gordan_tensor_amd import api
    from clebsch_gordan_tensor_amd import synth as S

    api.lib()  # fails loudly when the HIP library is missing
    t0 = time.time()
    p = S.make_conv(args.config)
    g = p.graph
    N, E, C, P = g.n_nodes, g.n_edges, p.channels, p.n_paths
    log(f"[bench] {args.config}: N={N} E={E} C={C} P={P} dtype={p.dtype} "
        f"(generated in {time.time() - t0:.1f} s)")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    tdt = torch.bfloat16 if p.dtype == "bf16" else torch.float32
    up = lambda a, dt=None: (torch.from_numpy(np.ascontiguousarray(a)).to(dev)
                             if dt is None else torch.from_numpy(a).to(dev).to(dt))
    rowptr, sender, ev = up(g.rowptr), up(g.sender), up(g.evec)
    x, w, dm = up(p.x, tdt), up(p.w, tdt), up(p.dm, tdt)
    d = api.Desc(p.x_irreps, p.y_irreps, p.out_irreps, C)
    dx_, dy_, dout_ = d.dx, d.dy, d.dout
    m = torch.empty((N, dout_, C), device=dev, dtype=tdt)
    dxo = torch.empty((N, dx_, C), device=dev, dtype=tdt)
    dwo = torch.empty((E, P, C), device=dev, dtype=tdt)
    dYo = torch.empty((E, dy_), device=dev, dtype=torch.float32)
    ws = torch.empty(api.workspace_size(N, E), device=dev, dtype=torch.uint8)
    torch.cuda.synchronize()

    stream = torch.cuda.current_stream()
    ep0, ep1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    ep0.record(stream)
    api.conv_prepare_transpose(rowptr, sender, ws, edge_vec=ev)
    ep1.record(stream)
    torch.cuda.synchronize()
    prepare_ms = ep0.elapsed_time(ep1)

    def step(evs=None):
        if evs:
            evs[0].record(stream)
        api.conv_forward(d, rowptr, sender, ev, x, w, out=m, workspace=ws)
        if evs:
            evs[1].record(stream)
        api.conv_backward(d, rowptr, sender, ws, ev, x, w, dm, dx=dxo, dw=dwo, dY=dYo)
        if evs:
            evs[2].record(stream)

    for _ in range(args.warmup):
        step()
    torch.cuda.synchronize()
    evs = [[torch.cuda.Event(enable_timing=True) for _ in range(3)] for _ in range(args.steps)]
    torch.cuda.synchronize()
    t_start = time.perf_counter()
    for i in range(args.steps):
        step(evs[i])
    torch.cuda.synchronize()
    wall_ms = (time.perf_counter() - t_start) * 1e3
    fwd_ms = np.array([e[0].elapsed_time(e[1]) for e in evs])
    bwd_ms = np.array([e[1].elapsed_time(e[2]) for e in evs])
    ms_per_step = wall_ms / args.steps
    log(f"[bench] fwd {fwd_ms.mean():.3f} ms  bwd {bwd_ms.mean():.3f} ms  "
        f"step {ms_per_step:.3f} ms  prepare (first call) {prepare_ms:.3f} ms")

    # the pages' protocol on the headline kernels: 100 individually timed runs
    fprot = protocol(lambda: api.conv_forward(d, rowptr, sender, ev, x, w, out=m, workspace=ws),
                     stream)
    bprot = protocol(lambda: api.conv_backward(d, rowptr, sender, ws, ev, x, w, dm, dx=dxo, dw=dwo,
                                               dY=dYo), stream)
    pprot = protocol(lambda: api.conv_prepare_transpose(rowptr, sender, ws, edge_vec=ev), stream,
                     runs=20, warm=2)
    log(f"[bench] protocol: fwd median {fprot['median_ms']:.3f} min {fprot['min_ms']:.3f} "
        f"fastest-20% {fprot['fastest20_mean_ms']:.3f} ms; bwd median {bprot['median_ms']:.3f} "
        f"min {bprot['min_ms']:.3f} fastest-20% {bprot['fastest20_mean_ms']:.3f} ms; prepare "
        f"median {pprot['median_ms']:.3f} ms")

    # achievable HBM rates with torch's own streaming kernels
    ceil = hbm_ceilings(dev, stream)
    copy_gbs = ceil["copy_gbs"]
    log(f"[bench] torch streams: read {ceil['read_gbs']:.0f}, copy {ceil['copy_gbs']:.0f}, "
        f"add {ceil['add_gbs']:.0f} GB/s")

    extras = {}
    if not args.no_extras:
        # the chain from dY to position gradients on the same graph (not part
        # of the step: the step is the convolution forward + backward)
        dvec = torch.empty((E, 3), device=dev, dtype=torch.float32)
        dpos = torch.empty((N, 3), device=dev, dtype=torch.float32)
        lmax = max(l for l, _ in p.y_irreps)

        def chain():
            api.spherical_harmonics_backward(lmax, ev, dYo, out=dvec)
            api.edge_grad_to_nodes(rowptr, sender, ws, dvec, out=dpos)

        extras["force_chain"] = time_call(chain, stream, 100)
        extras["force_chain"]["bytes"] = E * (12 + 4 * dy_ + 12) + E * 32 + N * 28
        del dvec, dpos
        extras.update(tp_measurements(api, S, dev, stream))
        extras.update(linear_measurement(api, S, p, dev, stream))
        extras.update(training_measurement(api, S, p, dev, stream))
        if p.dtype == "f32":
            extras.update(radial_measurement(api, d, g, rowptr, sender, ev, x, dwo, ws, dev,
                                             stream))

    esize = 2 if p.dtype == "bf16" else 4
    fwd_b, bwd_b = algorithmic_bytes(N, E, dx_, dy_, dout_, P, C, esize)
    bwd_gbs = bwd_b / (bwd_ms.mean() * 1e-3) / 1e9
    fwd_gbs = fwd_b / (fwd_ms.mean() * 1e-3) / 1e9
    step_gbs = (fwd_b + bwd_b) / (ms_per_step * 1e-3) / 1e9
    traffic = measured_traffic(args.config)
    # the backward's read:write mix (algorithmic: primals, dm and indices read;
    # dx, dw, dY written) and the rate torch's streams reach for that mix
    bwd_write = N * dx_ * C * esize + E * P * C * esize + E * dy_ * 4
    bwd_read = bwd_b - bwd_write
    mix = mix_ceiling_gbs(bwd_read, bwd_write, ceil)
    # the same for the counter-measured mix, and the backward's actual rate
    counter = None
    if traffic:
        counter = {"bytes": traffic["total"], "read": traffic["read"], "write": traffic["write"],
                   "gbs": traffic["total"] / (bwd_ms.mean() * 1e-3) / 1e9,
                   "mix_ceiling_gbs": mix_ceiling_gbs(traffic["read"], traffic["write"], ceil)}
    ff, bf = method_flops(api, d)

    configs, cpu_more = {}, {}
    if not args.no_configs and args.config == "mace64k":
        for name in ("tiny", "water3k", "ho20k"):
            rec, q = conv_record(api, S, name, dev, stream)
            configs[name] = rec
            if not args.no_cpu_baseline and name == "water3k":
                log("[bench] timing the fp64 oracle on water3k (all threads, then one) ...")
                cpu_more["water3k"] = cpu_full(q)
                cpu_more["water3k_single_thread"] = cpu_full(q, threads=1)
            if not args.no_cpu_baseline and name == "ho20k":
                log("[bench] timing the fp64 oracle on an ho20k sample ...")
                cpu_more["ho20k"] = cpu_baseline(q, 2000)
            del q

    cpu = None
    if not args.no_cpu_baseline:
        log("[bench] timing the fp64 oracle on a sample ...")
        cpu = cpu_baseline(p, CPU_SAMPLE_RECEIVERS)
        cpu["cpu_model"] = cpu_model()
        if cpu_more:
            cpu["other_workloads"] = cpu_more
        log(f"[bench] oracle {cpu['value']:.0f} edges/s on {cpu['cores']} threads")

    out = {
        "metric": "edges/sec and achieved HBM GB/s (% of peak), fused equivariant conv fwd+bwd",
        "value": E / (ms_per_step * 1e-3),
        "unit": "edges/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": ms_per_step,
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": p.dtype,
        "data": "synthetic (seeded uniform atoms, radius graph, N(0,1) features/weights/cotangent)",
        "config": {"workload": f"{args.config}: {N} atoms at 0.1/A^3, 5 A cutoff, {E} edges, "
                               f"x {C}x(" + "+".join(f"{l}{'e' if q > 0 else 'o'}" for l, q in p.x_irreps)
                               + "), Y l<=3, out " + f"{C}x("
                               + "+".join(f"{l}{'e' if q > 0 else 'o'}" for l, q in p.out_irreps)
                               + f"), {P} paths, fwd+bwd",
                   "n_nodes": N, "n_edges": E, "channels": C, "paths": P},
        "achieved_gbs_fwd_bwd": step_gbs,
        "hbm_frac_fwd_bwd": step_gbs / HBM_PEAK_GBS,
        "kernels": {
            "conv_forward": {"ms": float(fwd_ms.mean()), "bytes": fwd_b, "gbs": fwd_gbs,
                             "frac": fwd_gbs / HBM_PEAK_GBS, "protocol": fprot,
                             "tflops": ff * E * C / (fprot["median_ms"] * 1e-3) / 1e12},
            "conv_backward": {"ms": float(bwd_ms.mean()), "bytes": bwd_b, "gbs": bwd_gbs,
                              "frac": bwd_gbs / HBM_PEAK_GBS, "protocol": bprot,
                              "tflops": bf * E * C / (bprot["median_ms"] * 1e-3) / 1e12},
            # the first call on the graph: includes loading the prepare kernels' code
            "prepare_transpose_first_call_ms": prepare_ms,
            "prepare_transpose_per_graph_ms": pprot["median_ms"],
            "prepare_transpose_protocol": pprot,
            **extras,
        },
        "configs": configs,
        "device_copy_gbs": copy_gbs,
        "hbm_torch_streams_gbs": ceil,
        "hbm_mix_ceiling_gbs": mix,
        "roofline": {"kernel": "conv_backward", "bound": "hbm", "achieved": bwd_gbs,
                     "peak": HBM_PEAK_GBS, "unit": "GB/s", "frac": bwd_gbs / HBM_PEAK_GBS,
                     "traffic": traffic["total"] if traffic else None,
                     "mix_ceiling": mix, "frac_of_mix_ceiling": bwd_gbs / mix,
                     "counter_measured": counter},
        "cpu_baseline": cpu,
    }
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
