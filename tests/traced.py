"""Which kernels a call launches, for tests that have to reach a certain one."""

import paged_kv_cache_46_gb300 as ts


def kernels_of(call):
    """(the call's result, names of the kernels it launched in order)."""
    ts.ts_trace_collect()
    ts.ts_trace_enable(True)
    try:
        result = call()
    finally:
        ts.ts_trace_enable(False)
    return result, [name for name, _ in ts.ts_trace_collect()]
