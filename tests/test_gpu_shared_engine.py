"""The engine's decode graphs with shared_prefix: requests of two families with
a common system prompt each go through the scheduler's prefix cache, and their
decode steps read the common blocks once per group.  Every decode step of every
layer is checked against the oracle, the caches bit for bit at the end."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_125_gb300 as kvp
from paged_kv_cache_125_gb300 import workloads as W
from paged_kv_cache_125_gb300.engine_replay import EngineReplay
from paged_kv_cache_125_gb300.graphs import DecodeGraphs

from parity import BF16_NAN, assert_attn_close, assert_status_ok, run_oracle, u16
from test_gpu_shared_decode import plan_prefixes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (4, 2, 64)])
def test_engine_with_shared_prefixes(hq, hkv, d):
    layers, bs, nb = 2, 16, 260
    rng = np.random.default_rng(3)
    system = [rng.integers(0, 1 << 30, 200).tolist(), rng.integers(0, 1 << 30, 150).tolist()]
    requests = [(system[i % 3 // 2] + rng.integers(0, 1 << 30, 5 + 7 * i % 40).tolist(), 6 + 5 * i % 23)
                for i in range(24)]
    eng = EngineReplay(requests, layers, hq, hkv, d, bs, nb, 32, 2000, "cuda", shared_prefix=True)
    ora = [tuple(np.full((nb, bs, hkv, d), BF16_NAN, np.uint16) for _ in range(2)) for _ in range(layers)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    shared = steps = 0
    kvp.device_status()
    while not eng.done():
        st = eng.schedule()
        m, n = st.meta, st.num_new
        if st.is_prefill:
            q, k, v = (torch.randn((layers, n, h, d), generator=gen, device="cuda").to(torch.bfloat16)
                       for h in (hq, hkv, hkv))
            eng.launch(st, q, k, v)
        else:
            q, k, v = eng.decode_inputs(st)
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            out = eng.launch(st)
        torch.cuda.synchronize()
        assert_status_ok()
        for l, (kc, vc) in enumerate(ora):
            oracle.kv_store(k[l].cpu(), v[l].cpu(), m.slot_mapping, kc, vc)
            if not st.is_prefill:
                want = oracle.decode(q[l].cpu(), kc, vc, m.block_tables, m.context_lens, hq, hkv, d ** -0.5)
                assert_attn_close(out[l], want, f"step {steps} layer {l}")
        if not st.is_prefill:
            pb = eng.graphs.bucket(n)
            shared += sum(p > 0 for p in plan_prefixes(eng.graphs.plan, pb)[:n])
        eng.commit(st, [int(x) for x in rng.integers(0, 1 << 30, len(st.seq_ids))])
        steps += 1
    assert shared > 100, shared  # rows that read a prefix with their group, over the decode steps
    for l, (kc, vc) in enumerate(ora):
        gk, gv = eng.cache(l)
        assert np.array_equal(u16(gk), kc) and np.array_equal(u16(gv), vc), l


def test_bucketed_graphs_without_anything_shared():
    hq, hkv, d, bs, max_bs, max_blocks = 16, 8, 128, 32, 16, 9
    nb = max_bs * max_blocks + 2
    kc = torch.empty((nb, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    graphs = DecodeGraphs(kc, vc, hq, max_blocks, max_bs=max_bs, shared_prefix=True)
    rng = np.random.default_rng(bs)
    for b in (1, 3, 11, 16):
        w = W.decode_workload(f"b{b}", rng.integers(1, max_blocks * bs + 1, size=b).tolist(), hq, hkv, d, bs, nb)
        kc.fill_(float("nan"))
        vc.fill_(float("nan"))
        w.place_history(kc, vc)
        st, m = w.steps[0].store, w.steps[0].attn.meta
        out = graphs.run(w.steps[0].attn.q.cuda(), st.k.cuda(), st.v.cuda(), st.slot_mapping.cuda(),
                         m.block_tables.cuda(), m.context_lens.cuda())
        torch.cuda.synchronize()
        assert_status_ok()
        ref, kr, vr = run_oracle(w)
        assert np.array_equal(u16(kc), kr) and np.array_equal(u16(vc), vr), b
        assert_attn_close(out, ref[0], f"b={b}")
        assert torch.all(graphs.out[b:graphs.bucket(b)].float() == 0)
