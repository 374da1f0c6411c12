"""The scratch kept per (device, stream). On the CPU: its host logic
(csrc/scratch_cache.h) compiled against an allocator that only keeps books. On
the GPU: graphs captured with it replay the right results after other calls on
the stream needed more."""
import os
import subprocess

import pytest
import torch

import moe_ragged_contraction_gb300 as mx

CSRC = os.path.join(os.path.dirname(os.path.abspath(mx.__file__)), "csrc")

BOOKS = r"""
#include "scratch_cache.h"
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)
struct Books {
    char* next = reinterpret_cast<char*>(4096);
    std::map<void*, size_t> live;
    int fail = 0;
    int allocate(void** p, size_t n, int) {
        if (fail) return fail;
        *p = next; next += n; live[*p] = n; return 0;
    }
    int release(void* p, int) { return live.erase(p) ? 0 : 99; }
};
using mxw::Scratch;
int main() {
    Books a;
    mxw::ScratchCache<int, Books> c;
    void *p = nullptr, *q = nullptr, *r = nullptr;
    int e = 0;
    // one block a (device, stream), kept and reused
    CHECK(c.get(a, 0, 1, 100, false, &p, &e) == Scratch::ok && a.live.size() == 1);
    CHECK(c.get(a, 0, 1, 80, false, &q, &e) == Scratch::ok && q == p);
    CHECK(c.get(a, 0, 2, 80, false, &q, &e) == Scratch::ok && q != p);
    CHECK(c.get(a, 1, 1, 80, false, &r, &e) == Scratch::ok && r != p && r != q && a.live.size() == 3);
    // growth releases what no graph holds
    CHECK(c.get(a, 0, 2, 200, false, &r, &e) == Scratch::ok && !a.live.count(q) && a.live[r] == 200);
    // no growth under capture, no block for a new stream
    CHECK(c.get(a, 0, 1, 101, true, &q, &e) == Scratch::capturing);
    CHECK(c.get(a, 0, 3, 1, true, &q, &e) == Scratch::capturing && a.live.size() == 3);
    // a block that a graph was given stays, whatever later calls need
    CHECK(c.get(a, 0, 1, 100, true, &q, &e) == Scratch::ok && q == p);
    CHECK(c.get(a, 0, 1, 500, false, &r, &e) == Scratch::ok && r != p && a.live.count(p) && a.live[r] == 500);
    // the larger one was given to no graph
    CHECK(c.get(a, 0, 1, 900, false, &q, &e) == Scratch::ok && !a.live.count(r) && a.live.count(p));
    // graphs of two sizes: both blocks stay
    CHECK(c.get(a, 0, 1, 900, true, &r, &e) == Scratch::ok && r == q);
    CHECK(c.get(a, 0, 1, 1000, false, &r, &e) == Scratch::ok && a.live.count(p) && a.live.count(q) && a.live.count(r));
    // a failure is passed on and leaves a cache that works
    a.fail = 2;
    CHECK(c.get(a, 0, 1, 2000, false, &r, &e) == Scratch::failed && e == 2);
    CHECK(c.get(a, 0, 9, 10, false, &r, &e) == Scratch::failed && e == 2);
    a.fail = 0;
    CHECK(c.get(a, 0, 1, 10, false, &r, &e) == Scratch::ok && a.live[r] == 10);
    CHECK(c.get(a, 0, 9, 10, false, &r, &e) == Scratch::ok && a.live[r] == 10);
    CHECK(a.live.count(p) && a.live.count(q));
    puts("ok");
}
"""


def test_blocks_given_to_a_graph_are_kept(tmp_path):
    src, exe = tmp_path / "books.cc", tmp_path / "books"
    src.write_text(BOOKS)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
def test_graph_replays_after_the_scratch_has_grown():
    """The layer and a small and a large update on one stream: the graph of the first is replayed after the last has
    taken far more scratch and other streams' calls have had the memory that became free."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    E, H, I, T = 6, 512, 256, 20
    w13, s13 = mx.quantize_tokenwise(rand(E * 2 * I, H))
    w2, s2 = mx.quantize_tokenwise(rand(E * H, I))
    args = (rand(T, H).bfloat16(), rand(E, H).bfloat16(), w13.view(E, 2 * I, H), s13.view(E, 2 * I, -1), w2.view(E, H, I), s2.view(E, H, -1), 3)
    g, big = rand(2, 264, 520), rand(8, 1024, 1040)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want = mx.moe_layer(*args), mx.muon_update(g)
    stream.synchronize()
    outs = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        mx.moe_layer(*args, out=outs[0])
        mx.muon_update(g, out=outs[1])
    others = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(2):
        with torch.cuda.stream(stream):
            mx.muon_update(big)
        stream.synchronize()
        for s in others:  # scratch of the sizes that were in use before
            with torch.cuda.stream(s):
                assert torch.equal(mx.muon_update(g), want[1])
                mx.muon_update(big)
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert mx.device_status(clear=True) == 0
