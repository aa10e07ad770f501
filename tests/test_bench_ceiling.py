"""bench.py's MMA-only ceiling is taken with the GPU rested (fakes, no GPU)."""
import importlib.util
import os
import types

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench():
    spec = importlib.util.spec_from_file_location("bench_module", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_ceiling_is_not_the_power_capped_one(monkeypatch):
    """A fake GPU, hot from dense work: it runs the loop at 3150 TOPS until it has
    rested 0.3 s, then at 4550, the first launch of a kernel slower."""
    bench = _bench()
    clock = {"now": 0.0, "first": True}
    monkeypatch.setattr(bench.time, "sleep", lambda s: clock.update(now=clock["now"] + s))

    def launch(pair, k_blocks):
        tops = 3150e12 if clock["now"] < 0.3 else 430e12 if clock["first"] else 4550e12
        clock["first"] = False
        clock["now"] += 148 * k_blocks * 4 * 2.0 * 128 * 256 * 32 / tops
        return 148

    class Event:
        def __init__(self, enable_timing):
            pass

        def record(self, stream):
            self.at = clock["now"]

        def elapsed_time(self, other):
            return (other.at - self.at) * 1e3

    cuda = types.SimpleNamespace(Event=Event, current_stream=lambda: None, synchronize=lambda: None)
    hq = types.SimpleNamespace(hq_debug_mma_ceiling=launch)
    got = bench.measure_mma_ceiling(hq, types.SimpleNamespace(cuda=cuda))
    for name in ("single_cta_TOPS", "cta_pair_TOPS"):
        assert abs(got[name] - 4550.0) < 1.0, (name, got)
