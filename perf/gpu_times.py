"""GPU time of the calls that perf/more_operators.py lists: each in a captured graph of calls that go round over three
sets of inputs (as many calls as take some 2 ms, 12 at least), nine replays timed by events, least and median per
call.

    python perf/gpu_times.py [part of a case's name ...]

What a call takes through the binding is more where the GPU is done before the host (some 10 us a call).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from perf import more_operators as cases  # noqa: E402

REPLAYS = 9


def replays(states, calls):
    """Times of a call in us, one for each replay of a graph of so many calls."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(calls):
            cases.run(states[i % len(states)])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    times = []
    for _ in range(REPLAYS):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / calls)
    return sorted(times)


def gpu_time(case):
    """Least and median time of a call in us."""
    states = [cases.prepare(case, seed) for seed in range(3)]
    for state in states:
        cases.run(state)
    torch.cuda.synchronize()
    times = replays(states, max(12, min(300, round(2000 / replays(states, 12)[0]))))
    return times[0], times[REPLAYS // 2]


def main(parts):
    cases.own = True
    for case in cases.listed():
        if not parts or any(part in case["name"] for part in parts):
            least, median = gpu_time(case)
            print(f"{case['name']:<20} least {least:8.2f} us  median {median:8.2f} us", flush=True)


if __name__ == "__main__":
    main(sys.argv[1:])
