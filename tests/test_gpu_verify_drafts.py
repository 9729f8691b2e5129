"""GPU: the verification of drafted tokens against the definition, request by request."""
import pytest
import torch

import ssm_reference as ref
import stream_compaction_decoupled_gb300 as gb

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def inputs(b, k, v, dtype, seed, lookup=False, ids=torch.int64, pad=0, near=0.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((b, k + 1, v), generator=g) * 2
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :k] + near * torch.randn((b, k, v), generator=g), -1)
    drafts = torch.multinomial(q.reshape(b * k, v), 1, generator=g).view(b, k) if k else torch.zeros((b, 0), dtype=torch.int64)

    def rows(m):
        if not pad:
            return m.to(dtype).cuda()
        buf = torch.full((*m.shape[:2], m.shape[2] + pad), 3.0, dtype=dtype, device="cuda")
        buf[..., pad:] = m.to(dtype)
        return buf[..., pad:]

    return {"drafts": drafts.to(ids).cuda(), "target": rows(p), "draft": None if lookup else rows(q),
            "accept": torch.rand((b, k), generator=g).cuda(), "sample": torch.rand((b,), generator=g).cuda()}


def check(args, lengths=None):
    got = gb.verify_drafts(**args, lengths=lengths)
    accepted, tokens = ref.verify(**args, lengths=lengths)
    assert got.accepted.dtype == got.tokens.dtype == torch.int32
    assert torch.equal(got.accepted.cpu(), accepted)
    assert torch.equal(got.tokens.cpu(), tokens)
    return got


@pytest.mark.parametrize("lookup", [False, True], ids=["drafter", "lookup"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 0, 50), (3, 2, 7), (5, 4, 257), (2, 40, 300), (7, 3, 5000), (33, 5, 1024),
                                  (2, 2, 50021), (4, 3, 128000), (700, 1, 64)], ids=str)
def test_verify(size, dt, lookup):
    check(inputs(*size, DT[dt], sum(size), lookup))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_rows_of_every_alignment_and_int32_drafts(dt, pad):
    check(inputs(4, 3, 1003, DT[dt], pad, pad=pad, ids=torch.int32))
    check(inputs(4, 3, 1024, DT[dt], pad, pad=pad, lookup=True))


def test_lengths():
    args = inputs(9, 6, 500, torch.float32, 1, near=0.05)
    lengths = torch.tensor([0, 1, 2, 3, 4, 5, 6, 0, 6], dtype=torch.int32, device="cuda")
    got = check(args, lengths)
    assert (got.accepted.cpu() <= lengths.cpu()).all() and int(got.accepted.max()) > 3
    lengths[0], lengths[1] = -3, 99
    check(args, lengths)
    assert gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK


def test_every_place_of_the_draw():
    """Probabilities that are powers of two: each border is exact, a draw at one goes to the next."""
    v = 4096
    p = torch.zeros((v + 1, 1, v), device="cuda")
    p[:, 0] = 1.0 / v
    sample = (torch.arange(v + 1).float() / v).cuda()
    sample[v] = 1.0 - 2.0 ** -24
    args = {"drafts": torch.zeros((v + 1, 0), dtype=torch.int64, device="cuda"), "target": p, "draft": None,
            "accept": torch.zeros((v + 1, 0), device="cuda"), "sample": sample}
    got = gb.verify_drafts(**args)
    assert torch.equal(got.tokens[:, 0].cpu(), torch.cat([torch.arange(v), torch.tensor([v - 1])]).int())


def test_sums_as_in_64_bits():
    """A large probability first and many small ones behind it: in fp32 the small ones would be
    lost one by one."""
    v, b = 200000, 64
    p = torch.full((b, 1, v), 1e-9, device="cuda")
    p[:, 0, 0] = 0.9
    sample = torch.linspace(0.9995, 0.999999, b).cuda()
    args = {"drafts": torch.zeros((b, 0), dtype=torch.int64, device="cuda"), "target": p, "draft": None,
            "accept": torch.zeros((b, 0), device="cuda"), "sample": sample}
    got = check(args)
    # The small ones hold 2e-4 of 0.9002: the samples above 1 - 2.22e-4 fall among them, (0.999999 -
    # 0.999778) / (0.999999 - 0.9995) = 0.44 of all, each 7135 values from the next.
    assert len(set(got.tokens[:, 0].tolist())) > int(0.43 * b)


def test_rows_with_nothing_left_and_odd_probabilities():
    args = inputs(6, 2, 100, torch.float32, 4)
    args["target"][0] = 0.0                      # nothing can be drawn
    args["target"][1] = args["target"][1] * 0 - 1  # negative: as zero
    args["target"][2, :, 50:] = float("nan")
    args["draft"][3] = float("nan")              # as zero: everything is accepted
    args["target"][4, 0] = args["draft"][4, 0]   # equal: accepted
    args["accept"][5] = 0.0
    args["target"][5, 0, int(args["drafts"][5, 0])] = 0.0  # impossible: refused even so
    got = check(args)
    assert got.tokens[0].tolist() == [-1, -1, -1] and int(got.accepted[5]) == 0
    args["drafts"][4, 0] = 100
    args["drafts"][5, 1] = -7
    got = check(args)
    assert int(got.accepted[4]) == 0 and gb.device_error() == gb.ERR_RANGE and gb.device_error() == gb.OK


def test_a_refused_lookup_is_not_drawn():
    b, v = 64, 40
    args = inputs(b, 1, v, torch.float32, 5, lookup=True)
    args["accept"][:] = 1.0 - 2.0 ** -24
    got = check(args)
    assert not (got.tokens[:, 0].cpu() == args["drafts"][:, 0].cpu().int())[got.accepted.cpu() == 0].any()
    args["target"][0] = 0.0
    args["target"][0, 0, int(args["drafts"][0, 0])] = 0.5  # the refused token had all there was
    assert gb.verify_drafts(**args).tokens[0].tolist() == [-1, -1]


def test_what_is_drawn_is_distributed_as_the_target():
    """Over all random numbers the first token is distributed as the target's first row, whatever
    the drafter's: counts of 40000 draws within six standard deviations."""
    b, v = 40000, 5
    g = torch.Generator().manual_seed(8)
    p = torch.tensor([0.5, 0.2, 0.15, 0.1, 0.05])
    q = torch.tensor([0.1, 0.5, 0.2, 0.1, 0.1])
    args = {"drafts": torch.multinomial(q, b, True, generator=g).view(b, 1).cuda(),
            "target": p.expand(b, 2, v).contiguous().cuda(), "draft": q.expand(b, 1, v).contiguous().cuda(),
            "accept": torch.rand((b, 1), generator=g).cuda(), "sample": torch.rand((b,), generator=g).cuda()}
    first = gb.verify_drafts(**args).tokens[:, 0].cpu().long()
    counts = torch.bincount(first, minlength=v).double()
    assert ((counts - b * p.double()).abs() <= 6 * (b * p.double() * (1 - p.double())).sqrt()).all()


def test_streams_graphs_and_broadcast_rows():
    args = inputs(6, 3, 3001, torch.bfloat16, 6)
    want = gb.verify_drafts(**args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gb.verify_drafts(**args, stream=side)
    side.synchronize()
    assert torch.equal(got.tokens, want.tokens) and torch.equal(got.accepted, want.accepted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gb.verify_drafts(**args)
    held.tokens.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held.tokens, want.tokens)
    args["target"] = args["target"][:1].expand(6, -1, -1)
    args["draft"] = args["draft"][:1].expand(6, -1, -1)
    check(args)


def test_refusals():
    args = inputs(3, 2, 50, torch.float32, 7)
    for bad in (dict(drafts=args["drafts"].float()), dict(draft=args["draft"].half()), dict(target=args["target"].double()),
                dict(accept=args["accept"].double())):
        with pytest.raises(TypeError):
            gb.verify_drafts(**{**args, **bad})
    for bad in (dict(drafts=args["drafts"][:, :1]), dict(draft=args["draft"][:, :1]), dict(sample=args["sample"][:2]),
                dict(target=args["target"][:, :0]), dict(target=args["target"][..., ::2]), dict(accept=args["accept"].cpu()),
                dict(lengths=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            gb.verify_drafts(**{**args, **bad})
