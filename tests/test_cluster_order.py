"""A CTA of a cluster may touch another's shared memory only once that one runs, which a barrier of the cluster says. Nothing on
a GPU shows a missing one as long as the CTAs happen to start together, so the sources are read: in every function that
reaches into another CTA, a barrier of the cluster has been waited for before the first access."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "bit_quantized_moe_gb300" / "csrc"
REACH = ("map_shared_rank", "leader_addr", "peer_addr", "pair_leader", "ld_cluster", "ld_cluster4")   # what makes or uses a peer's address
ACCESS = re.compile(r"\b(?:%s)\s*[<(]" % "|".join(REACH))
BARRIER = re.compile(r"\bcluster_sync_all\s*\(|\bcluster\.sync\s*\(|\bbarrier_wait\s*\(")


def functions(text):
    """(name, text) of each device function."""
    text = re.sub(r"//[^\n]*", "", text)
    starts = [m.start() for m in re.finditer(r"^(?=[^\s#]).*\b__(?:global|device)__\b", text, re.M)]
    for a, b in zip(starts, starts[1:] + [len(text)]):
        body = text[a:b]
        head = body[:body.index("{")] if "{" in body else body
        names = [n for n in re.findall(r"\b(\w+)\s*\(", head) if not n.startswith("__")]
        yield (names[0] if names else ""), body


def unordered(text):
    """Functions whose first access to another CTA's shared memory no barrier precedes."""
    bad = []
    for name, body in functions(text):
        first = ACCESS.search(body)
        if first and name not in REACH and not BARRIER.search(body[:first.start()]):
            bad.append(name)
    return bad


@pytest.mark.parametrize("path", sorted(p.name for p in CSRC.glob("*.cu*")))
def test_peers_run_before_their_memory_is_touched(path):
    assert unordered((CSRC / path).read_text()) == []


def test_the_reading_finds_what_it_looks_for():
    store = "__global__ void k(int a) {\n  if (a) cluster.map_shared_rank(x, 0)[0] = 1;\n  cluster.sync();\n}\n"
    assert unordered(store) == ["k"]
    assert unordered(store.replace("if (a)", "cluster.sync();\n  if (a)")) == []
    assert unordered(store.replace("if (a)", "auto t = cluster.barrier_arrive();\n  if (a)")) == ["k"]
    assert unordered("__device__ __forceinline__ int peer_addr(int a) {\n  return a;\n}\n" + store) == ["k"]
    found = {n for p in CSRC.glob("*.cu*") for n, body in functions(p.read_text()) if ACCESS.search(body) and n not in REACH}
    assert {"balance_finish_kernel", "b128_pair_kernel", "b128_few_kernel", "moe_sort_kernel", "mx_gemm_kernel"} <= found
