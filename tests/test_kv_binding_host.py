"""The native marshalling of the key-value cache's calls on a host without a GPU: what it
raises for tensors of the wrong extents, types and devices, and for tensors without
memory behind them (fake CUDA tensors, in a process of their own)."""
from test_binding_host import child


def test_malformed_tensors_raise():
    lines = child("""
    I32, BF = torch.int32, torch.bfloat16
    def cache(p=4, h=2, page=32, d=64):
        kv = [fake(p, h, page, d, dtype=S8) for _ in range(2)]
        return q.KvCache(*kv, *(fake(p, h, page // 16, dtype=U8) for _ in range(2)))
    c, t, n, st = cache(), fake(3, 5, dtype=I32), fake(3, dtype=I32), fake(4, dtype=I32)
    k = fake(7, 2, 64)
    app = lambda c=c, k=k, v=k, t=t, n=n, st=st, **kw: q.qmm_kv_append(c, k, v, t, n, starts=st, stream=S, **kw)
    att = lambda x=fake(7, 4, 64), c=c, t=t, n=n, st=st, **kw: q.qmm_kv_attention(x, c, t, n, starts=st, stream=S, **kw)
    rd = lambda c=c, t=t, n=n, st=st, rows=7, **kw: q.qmm_kv_read(c, t, n, starts=st, rows=rows, stream=S, **kw)
    cs = fake(9, 16)
    for name, f in {
        "value error": lambda: app(v=fake(7, 2, 63)),
        "other heads": lambda: app(k=fake(7, 3, 64), v=fake(7, 3, 64)),
        "other dim": lambda: app(k=fake(7, 2, 32), v=fake(7, 2, 32)),
        "flat k": lambda: app(k=fake(7, 128), v=fake(7, 128)),
        "half k": lambda: app(k=fake(7, 2, 64, dtype=torch.float16), v=fake(7, 2, 64, dtype=torch.float16)),
        "two types": lambda: app(v=fake(7, 2, 64, dtype=BF)),
        "gaps": lambda: app(k=fake(7, 2, 128)[..., ::2]),
        "scale shape": lambda: app(c=c._replace(k_exp=fake(4, 2, 1, dtype=U8))),
        "cache gaps": lambda: app(c=c._replace(v=fake(4, 2, 32, 128, dtype=S8)[..., ::2])),
        "cache type": lambda: app(c=c._replace(k=fake(4, 2, 32, 64, dtype=U8))),
        "table type": lambda: app(t=fake(3, 5, dtype=torch.int64)),
        "table flat": lambda: app(t=fake(3, dtype=I32)),
        "lengths": lambda: app(n=fake(4, dtype=I32)),
        "starts": lambda: app(st=fake(3, dtype=I32)),
        "no starts": lambda: app(st=None),
        "cos alone": lambda: app(cos=cs),
        "cos shape": lambda: app(cos=cs, sin=fake(9, 8)),
        "cos type": lambda: app(cos=cs.to(BF), sin=cs.to(BF)),
        "q rows": lambda: app(q=fake(6, 4, 64)),
        "q type": lambda: app(q=fake(7, 4, 64, dtype=BF)),
        "q none": lambda: app(q=fake(7, 0, 64)),
        "q_out alone": lambda: app(q_out=fake(7, 4, 64)),
        "q_out shape": lambda: app(q=fake(7, 4, 64), q_out=fake(7, 2, 64)),
        "device": lambda: app(t=fake(3, 5, dtype=I32, device="cuda:1")),
        "att dim": lambda: att(x=fake(7, 4, 128)),
        "att type": lambda: att(x=fake(7, 4, 64, dtype=S8)),
        "att out": lambda: att(out=fake(7, 4, 64, dtype=BF)),
        "att workspace": lambda: att(out=fake(7, 4, 64), workspace="no"),
        "att workspace gaps": lambda: att(out=fake(7, 4, 64), workspace=fake(10, dtype=U8).expand(5, 10)),
        "read out": lambda: rd(k_out=fake(6, 2, 64)),
        "read types": lambda: rd(k_out=fake(7, 2, 64), v_out=fake(7, 2, 64, dtype=BF)),
        "read type": lambda: rd(out_dtype=torch.float16),
        "read rows": lambda: rd(rows=-1),
        "read starts": lambda: rd(st=None),
    }.items():
        print(name + ":", outcome(f))
    """)
    assert len(lines) == 34
    for line in lines:
        assert ": ValueError: " in line, line


def test_tensors_without_memory_raise():
    lines = child("""
    I32 = torch.int32
    c = q.KvCache(*(fake(4, 2, 32, 64, dtype=S8) for _ in range(2)), *(fake(4, 2, 2, dtype=U8) for _ in range(2)))
    t, n = fake(3, 5, dtype=I32), fake(3, dtype=I32)
    x, o = fake(2, 3, 2, 64), fake(2, 3, 2, 64)
    print("append", outcome(torch.vmap(lambda k: q.qmm_kv_append(c, k, k, t, n, stream=S)), x))
    print("attention", outcome(torch.vmap(lambda k, o: q.qmm_kv_attention(k, c, t, n, out=o, stream=S)), x, o))
    print("read", outcome(torch.vmap(lambda k, v: q.qmm_kv_read(c, t, n, k_out=k, v_out=v, out_dtype=F32, stream=S)), x, o))
    """)
    assert len(lines) == 3
    for line in lines:
        assert line.split()[1] == "RuntimeError:", line
