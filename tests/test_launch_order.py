"""Calls of several launches that hand over through the scratch of their (device,
stream), made by several host threads on one stream. On the CPU: the lock that a call
holds from the lookup of its scratch to its last launch (csrc/scratch_cache.h), on a
stream that only keeps a list. On the GPU: each call gets its own results."""
import os
import subprocess
import threading

import pytest
import torch

import moe_ragged_contraction_gb300 as mx

CSRC = os.path.join(os.path.dirname(os.path.abspath(mx.__file__)), "csrc")

THREADS = r"""
#include "scratch_cache.h"
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <utility>
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)
// What is enqueued on a stream, in order: (call, step), step 0 a release, 1 .. 3 the launches.
std::mutex mu;
std::vector<std::pair<int, int>> queue[2];
void enqueue(int stream, int call, int step) {
    std::this_thread::yield();
    std::lock_guard<std::mutex> lk(mu);
    queue[stream].push_back({call, step});
}
struct Books {
    int call = 0;
    char* next = reinterpret_cast<char*>(4096);
    int allocate(void** p, size_t n, int) { *p = next; next += n; return 0; }
    int release(void*, int stream) { enqueue(stream, call, 0); return 0; }
};
int main() {
    mxw::StreamLocks<int> locks;
    mxw::ScratchCache<int, Books> cache;
    std::mutex cache_mu;
    Books books;
    std::atomic<int> calls{0};
    auto work = [&](int me) {
        for (int i = 0; i < 400; ++i) {
            const int call = calls++, stream = me & 1;
            std::unique_lock<std::mutex> launches = locks.hold(0, stream);
            {
                std::lock_guard<std::mutex> lk(cache_mu);
                books.call = call;
                void* p;
                int e;
                CHECK(cache.get(books, 0, stream, 100 + call, false, &p, &e) == mxw::Scratch::ok);  // (mostly more than before)
            }
            for (int s = 1; s <= 3; ++s) enqueue(stream, call, s);
        }
    };
    std::vector<std::thread> ts;
    for (int t = 0; t < 8; ++t) ts.emplace_back(work, t);
    for (auto& t : ts) t.join();
    for (auto& q : queue) {
        // a call's launches are neighbours: nobody else's come between them, and no release
        size_t at = 0, n = 0;
        for (; at < q.size(); ++n) {
            const int call = q[at].first;
            if (q[at].second == 0) ++at;
            for (int s = 1; s <= 3; ++s, ++at) CHECK(at < q.size() && q[at] == std::make_pair(call, s));
        }
        CHECK(n == 1600);
    }
    // a stream's lock holds up no other stream and no other device
    auto a = locks.hold(0, 0);
    auto b = locks.hold(0, 1);
    auto c = locks.hold(1, 0);
    std::thread([&] { auto d = locks.hold(2, 0); CHECK(d.owns_lock()); }).join();
    // and is the same one at each call
    std::atomic<bool> got{false};
    std::thread other([&] { auto d = locks.hold(0, 0); got = true; });
    std::this_thread::sleep_for(std::chrono::milliseconds(50));
    CHECK(!got);
    a.unlock();
    other.join();
    CHECK(got);
    puts("ok");
}
"""


def test_launches_of_a_call_are_neighbours(tmp_path):
    src, exe = tmp_path / "threads.cc", tmp_path / "threads"
    src.write_text(THREADS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def in_threads(calls, rounds):
    """Each call again and again in a thread of its own, all on one stream: the results of the last rounds."""
    start, got, errors = threading.Barrier(len(calls)), [[] for _ in calls], []

    def work(i):
        try:
            start.wait()
            for _ in range(rounds):
                got[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    return got


@pytest.fixture
def gen():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    yield g
    assert mx.device_status(clear=True) == 0


def check(calls, rounds=60):
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for mine, w in zip(in_threads(calls, rounds), want):
        for r in mine:
            assert all(torch.equal(a, b) for a, b in zip(r, w))


@pytest.mark.gpu
@pytest.mark.parametrize("own_stream", [False, True])
def test_norm_and_clipping_of_several_threads_on_one_stream(gen, own_stream):
    """Lists of different strength and length: few and many tensors, so that the stream's scratch grows, too."""
    stream = torch.cuda.Stream() if own_stream else None
    lists = [[torch.randn(n, generator=gen, device="cuda") * 4.0 ** i for _ in range(m)] for i, (n, m) in enumerate(((70001, 2), (33, 40), (5000, 200), (600000, 5)))]
    many = [torch.randn(3, generator=gen, device="cuda") for _ in range(2100)]
    torch.cuda.synchronize()

    def call(grads):
        outs = [torch.empty_like(g) for g in grads]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        return [mx.clip_grads(grads, 1.0, out=outs, stream=stream), mx.grad_norm(grads, stream=stream), *outs]

    check([lambda g=g: call(g) for g in (*lists, many)], 25)


@pytest.mark.gpu
def test_products_updates_and_layers_of_several_threads_on_one_stream(gen):
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731

    def gradient(E, N, K, M):
        (A, sA), (B, sB) = mx.quantize_tokenwise(rand(N, M)), mx.quantize_tokenwise(rand(K, M))
        offs = (torch.arange(1, E + 1, device="cuda") * (M // E // 32 * 32)).int()
        return lambda: [mx.wgrad_grouped(A, sA, B, sB, offs)]

    def product(E, N, K, M):
        X, sX = mx.quantize_tokenwise(rand(M, K))
        W, sW = mx.quantize_tokenwise(rand(E * N, K))
        offs = (torch.arange(1, E + 1, device="cuda") * (M // E)).int()
        return lambda: [mx.grouped_gemm(X, sX, W.view(E, N, K), sW.view(E, N, -1), offs)]

    def update(*shape):
        g = rand(*shape)
        return lambda: [mx.muon_update(g)]

    def layer(T, E, H, I):
        w13, s13 = mx.quantize_tokenwise(rand(E * 2 * I, H))
        w2, s2 = mx.quantize_tokenwise(rand(E * H, I))
        args = (rand(T, H).bfloat16(), rand(E, H).bfloat16(), w13.view(E, 2 * I, H), s13.view(E, 2 * I, -1), w2.view(E, H, I), s2.view(E, H, -1), 2)
        return lambda: [mx.moe_layer(*args)]

    calls = [gradient(4, 256, 128, 1024), gradient(7, 128, 512, 4096), product(5, 128, 256, 700), product(3, 512, 128, 2000), update(3, 264, 520), update(1, 512, 512),
             layer(20, 6, 512, 256), layer(3, 9, 256, 128)]
    torch.cuda.synchronize()
    check(calls)


def test_per_thread_streams_are_told_apart():
    """cudaStreamPerThread is one handle for a stream of each thread: the cache asks for the stream's number."""
    with open(os.path.join(CSRC, "abi.cu")) as f:
        text = f.read()
    assert "stream == cudaStreamPerThread" in text and "cudaStreamGetId(stream, &key.number)" in text
    assert "ScratchCache<cudaStream_t" not in text and "StreamLocks<cudaStream_t" not in text


@pytest.mark.gpu
def test_per_thread_streams(gen):
    """Updates of different threads on their own default streams, at once: as many scratch blocks."""
    stream = torch.cuda.ExternalStream(2)  # cudaStreamPerThread
    grads = [torch.randn((2, 264 + 8 * i, 520), generator=gen, device="cuda") for i in range(4)]
    want = [mx.muon_update(g) for g in grads]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    norms = [[torch.empty((), device="cuda") for _ in range(20)] for _ in grads]
    total = [mx.grad_norm([g]) for g in grads]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(grads)), []

    def work(i):
        try:
            start.wait()
            for o, n in zip(outs[i], norms[i]):
                mx.muon_update(grads[i], out=o, stream=stream)
                mx.grad_norm([grads[i]], out=n, stream=stream)
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(grads))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w, mine, n, norm in zip(want, outs, total, norms):
        assert all(torch.equal(o, w) for o in mine) and all(float(v) == float(n) for v in norm)


@pytest.mark.gpu
def test_entry_without_allocation_of_several_threads(gen):
    import ctypes

    lib = mx.load()
    f = lib.mxfp8_wgrad_grouped_noalloc
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    f.argtypes, f.restype = [P, P, P, P, P, I, I, I, L, P, P], I
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream

    def gradient(E, N, K, M):
        (A, sA), (B, sB) = mx.quantize_tokenwise(rand(N, M)), mx.quantize_tokenwise(rand(K, M))
        offs = (torch.arange(1, E + 1, device="cuda") * (M // E // 32 * 32)).int()

        def call():
            out = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
            assert f(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), offs.data_ptr(), E, N, K, M, out.data_ptr(), stream) == 0
            return [out]
        return call

    calls = [gradient(4, 256, 128, 1024), gradient(7, 128, 512, 4096), gradient(1, 64, 64, 64), gradient(3, 512, 256, 2048)]
    torch.cuda.synchronize()
    check(calls)
